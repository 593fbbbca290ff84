"""The operators around and beside the recurrence against their plain forms in 64 bits."""
import itertools

import pytest
import torch

from tests import recurrent_reference as ref

pytestmark = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
DEV = "cuda"


@pytest.fixture(scope="module")
def gdn():
    import gated_delta_rule_17_gb300 as gdn

    gdn.load()
    return gdn


def rand(gen, *shape, dtype=torch.float32, scale=1.0):
    return (scale * torch.randn(shape, generator=gen, device=DEV)).to(dtype)


def wide(gen, rows, width, dtype, pad):
    """Rows that are slices of longer ones."""
    return rand(gen, rows, width + pad, dtype=dtype)[:, pad:]


def near(got, want, bound, what):
    off = (got.double() - want).abs()
    bad = ~(off <= bound)
    assert not bad.any(), (what, int(bad.sum()), float((off / bound.clamp(min=1e-300)).max()), torch.nonzero(bad)[:4].tolist())


def offsets(lens):
    return [0] + list(itertools.accumulate(lens))


def batch(lens, packed):
    """The batch's arguments; a dense one where the lengths are alike."""
    cu = offsets(lens)
    if packed:
        return dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=DEV))
    return dict(B=len(lens), T=lens[0])


def make_conv(lens, D, width, dtype, pad=0, state=True, bias=True, seed=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rows = sum(lens)
    return dict(x=wide(gen, rows, D, dtype, pad), w=rand(gen, D, width, scale=0.5), b=rand(gen, D) if bias else None,
                h0=rand(gen, len(lens), width - 1, D, dtype=dtype) if state else None, dout=wide(gen, rows, D, dtype, pad),
                dST=rand(gen, len(lens), width - 1, D, dtype=dtype) if state else None, dtype=dtype)


def conv_error(y, mags, out, dtype):
    """Of the sum of the products: width + 1 roundings of its terms; silu's slope is at most 1.1, its exponential and division
    cost (|y| + 6) / 2 steps."""
    return 1.1 * 6 * ref.U * mags + (y.abs() + 6) * ref.U * out.abs() + ref.half(dtype) * out.abs() + ref.least(dtype)


CONV = [  # lengths, D, width, type, padding of a row, packed, state, bias
    ([1], 8, 2, "bf16", 0, False, True, True), ([1] * 5, 1112, 4, "bf16", 0, False, True, True), ([3] * 7, 264, 4, "fp16", 8, False, True, True),
    ([2], 256, 3, "fp32", 0, False, False, False), ([0, 1, 2, 3, 4, 5, 0, 37, 0], 136, 4, "bf16", 24, True, True, True),
    ([130, 1, 0, 77], 72, 3, "fp32", 8, True, True, False), ([33] * 3, 520, 2, "fp16", 0, False, True, True),
    ([0, 0], 64, 4, "bf16", 0, True, True, True), ([700, 1501, 3, 1900], 4096, 4, "bf16", 0, True, True, True),
    ([1025] * 4, 4096, 4, "bf16", 128, False, True, True), ([5000], 1024, 3, "fp32", 0, False, False, True),
]


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("lens,D,width,type,pad,packed,state,bias", CONV)
def test_conv(gdn, lens, D, width, type, pad, packed, state, bias, silu):
    c = make_conv(lens, D, width, TYPES[type], pad, state, bias)
    y, want, last, mags = ref.conv(c["x"].double(), c["w"].double(), c["b"].double() if bias else None,
                                   c["h0"].double() if state else None, offsets(lens), silu)
    out = torch.full((sum(lens) + 2, D + 8), 7.0, dtype=c["dtype"], device=DEV)
    kept = c["h0"].clone() if state else None
    gdn.causal_conv(c["x"], c["w"], out[1:-1, :D], bias=c["b"], state=kept, silu=silu, **batch(lens, packed))
    gdn.check()
    near(out[1:-1, :D], want, conv_error(y, mags, want, c["dtype"]), "out")
    assert (out[0] == 7).all() and (out[-1] == 7).all() and (out[:, D:] == 7).all()
    if state:
        assert torch.equal(kept.double(), last)


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("lens,D,width,type,pad,packed,state,bias", CONV)
def test_conv_backward(gdn, lens, D, width, type, pad, packed, state, bias, silu):
    c = make_conv(lens, D, width, TYPES[type], pad, state, bias)
    cu = offsets(lens)
    leaf = {n: c[n].double().detach().clone().requires_grad_(True) for n in ("x", "w", "b", "h0") if c[n] is not None}
    y, out, last, mags = ref.conv(leaf["x"], leaf["w"], leaf.get("b"), leaf.get("h0"), cu, silu)
    total = (out * c["dout"].double()).sum() + ((last * c["dST"].double()).sum() if state else 0.0)
    total.backward()
    dx, dw, db = torch.full_like(c["x"].contiguous(), 7), torch.full_like(c["w"], 7), torch.full((D,), 7.0, device=DEV)
    dh0 = torch.full_like(c["h0"], 7) if state else None
    gdn.causal_conv_backward(c["x"], c["w"], c["dout"], dx, dw, db, bias=c["b"], h0=c["h0"], dST=c["dST"], dh0=dh0, silu=silu,
                             **batch(lens, packed))
    gdn.check()
    with torch.no_grad():
        # dy = dout silu'(y): slope up to 1.1, its own slope up to 0.5
        dy_off = c["dout"].double().abs() * ((y.abs() + 8) * 2 * ref.U + 0.5 * 6 * ref.U * mags) if silu else 0 * y
        dy = c["dout"].double().abs() * 1.1
        w = leaf["w"].abs()
        rows = sum(lens)
        off, mag = y.new_zeros(rows, D), y.new_zeros(rows, D)
        off_w, mag_w = y.new_zeros(D, width), y.new_zeros(D, width)
        off_h, mag_h = y.new_zeros(len(lens), width - 1, D), y.new_zeros(len(lens), width - 1, D)
        for s in range(len(lens)):
            n = lens[s]
            z = torch.cat([leaf["h0"][s] if state else y.new_zeros(width - 1, D), leaf["x"][cu[s]:cu[s + 1]]]).abs()
            e, m = y.new_zeros(n + width - 1, D), y.new_zeros(n + width - 1, D)
            for j in range(width):
                e[j:j + n] += w[:, j] * dy_off[cu[s]:cu[s + 1]]
                m[j:j + n] += w[:, j] * dy[cu[s]:cu[s + 1]]
                off_w[:, j] += (z[j:j + n] * dy_off[cu[s]:cu[s + 1]]).sum(0)
                mag_w[:, j] += (z[j:j + n] * dy[cu[s]:cu[s + 1]]).sum(0)
            if state:
                m[n:] += c["dST"][s].double().abs()
            off[cu[s]:cu[s + 1]], mag[cu[s]:cu[s + 1]] = e[width - 1:], m[width - 1:]
            off_h[s], mag_h[s] = e[:width - 1], m[:width - 1]
        h = ref.half(c["dtype"])
        near(dx, leaf["x"].grad, off + 6 * ref.U * mag + h * leaf["x"].grad.abs() + ref.least(c["dtype"]), "dx")
        near(dw, leaf["w"].grad, off_w + (rows + 8) * ref.U * mag_w + 1e-30, "dweight")
        if bias:
            near(db, leaf["b"].grad, dy_off.sum(0) + (rows + 8) * ref.U * dy.sum(0) + 1e-30, "dbias")
        if state:
            near(dh0, leaf["h0"].grad, off_h + 6 * ref.U * mag_h + h * leaf["h0"].grad.abs() + ref.least(c["dtype"]), "dh0")


def test_conv_backward_against_differences(gdn):
    """The gradients as slopes of the forward itself, in fp32."""
    lens, D, width = [5, 2, 9], 64, 4
    c = make_conv(lens, D, width, torch.float32, seed=3)

    def loss(x, w, b, h0):
        out, kept = torch.empty_like(x), h0.clone()
        gdn.causal_conv(x, w, out, bias=b, state=kept, **batch(lens, True))
        return float((out.double() * c["dout"].double()).sum() + (kept.double() * c["dST"].double()).sum())

    dx, dw, db, dh0 = torch.empty_like(c["x"]), torch.empty_like(c["w"]), torch.empty_like(c["b"]), torch.empty_like(c["h0"])
    gdn.causal_conv_backward(c["x"], c["w"], c["dout"], dx, dw, db, bias=c["b"], h0=c["h0"], dST=c["dST"], dh0=dh0, **batch(lens, True))
    args = dict(x=c["x"], w=c["w"], b=c["b"], h0=c["h0"])
    gen, step = torch.Generator(device=DEV).manual_seed(9), 2.0 ** -7
    size = float(c["dout"].abs().sum())
    for name, grad in (("x", dx), ("w", dw), ("b", db), ("h0", dh0)):
        along = torch.randn(grad.shape, generator=gen, device=DEV)
        up, down = (loss(**{**args, name: args[name] + sign * step * along}) for sign in (1, -1))
        slope, want = (up - down) / (2 * step), float((grad.double() * along.double()).sum())
        # the third derivative of the loss along `along` is at most a few times `size` x |along|^3; fp32 outputs: 2^-24 of them each
        reach = float(along.abs().max()) * (1.0 if name in ("b",) else 4.0)
        assert abs(slope - want) <= step ** 2 * size * reach ** 3 + size * 2 ** -22 / step, name


def ssm(lens, nk, nv, dk, dv, pad=0, seed=0, steps=0.05, rate=8.0, dt=torch.float32, skip=True, softplus=True):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    rows = sum(lens)
    bf = torch.bfloat16
    s = dict(q=wide(gen, rows, nk * dk, bf, pad), k=wide(gen, rows, nk * dk, bf, pad), v=wide(gen, rows, nv * dv, bf, pad))
    s["a"] = -rate * torch.rand(nv, generator=gen, device=DEV)
    target = steps * (0.2 + torch.rand(nv, generator=gen, device=DEV))
    s["bias"] = target + torch.log(-torch.expm1(-target)) if softplus else 0 * target
    s["dt"] = (rand(gen, rows, nv, scale=0.5) if softplus else target * torch.rand(rows, nv, generator=gen, device=DEV)).to(dt)
    s["skip"] = rand(gen, nv) if skip else None
    s["state"] = rand(gen, len(lens), nv, dk, dv, scale=0.3)
    z = s["dt"].double() + s["bias"].double()
    s["d"] = torch.nn.functional.softplus(z, threshold=1e4) if softplus else z
    s["args"] = dict(nk=nk, nv=nv, dk=dk, dv=dv, dt_bias=s["bias"], skip=s["skip"], softplus=softplus)
    return s


def ssm_want(s, lens):
    g = s["args"]
    nk, nv, dk, dv = g["nk"], g["nv"], g["dk"], g["dv"]
    zero = torch.zeros(nv, device=DEV, dtype=torch.float64)
    return ref.scan(s["q"].double().unflatten(1, (nk, dk)), s["k"].double().unflatten(1, (nk, dk)), s["v"].double().unflatten(1, (nv, dv)),
                    s["d"], s["a"].double(), s["skip"].double() if s["skip"] is not None else zero, s["state"].double(), offsets(lens), nv // nk)


def check_scan(out, state, want, rows):
    o, S, mags, M = want
    # Products in bf16, whose half step is 2^-8: A, f_hi and V', or S, each rounded once (3 x 2^-8 < 2^-6); the output itself by another
    near(out.view(o.shape), o, 2.0 ** -6 * mags + 2.0 ** -8 * o.abs() + 1e-30, "out")
    # The state's terms: f in two parts is off by 2^-8 x 2^-8; lo, at most 2 x 2^-8 of the term, is rounded by 2^-8 of itself: 2^-15.
    # Together 1.5 x 2^-15; fp32 sums and exponentials the rest of 2^-14
    near(state, S, 2.0 ** -14 * M + 1e-30, "state")
    if rows:
        # as sums of many terms they come much closer: three roundings of 2^-8 / sqrt(3) at most each, and the output's own: 4.5e-3
        assert float((out.view(o.shape).double() - o).norm()) <= 5e-3 * float(mags.norm())
        assert float((state.double() - S).norm()) <= 1e-5 * float(M.norm())


SCAN = [  # lengths, nk, nv, dk, dv, padding, packed
    ([1], 1, 1, 64, 64, 0, False), ([1] * 3, 1, 2, 128, 64, 0, False), ([127, 128, 129, 0, 1, 300], 2, 6, 128, 128, 8, True),
    ([5, 640, 0, 257], 1, 3, 128, 64, 24, True), ([333], 2, 10, 64, 64, 0, False), ([200] * 3, 3, 3, 64, 128, 0, False),
    ([0, 0, 7], 2, 4, 128, 64, 0, True), ([1500, 4, 900], 1, 5, 64, 64, 8, True), ([2048], 1, 2, 128, 128, 0, False),
]


@pytest.mark.parametrize("steps,rate", [(0.05, 8.0), (1.0, 4.0), (3.0, 30.0), (1e-4, 1e-3)])
@pytest.mark.parametrize("lens,nk,nv,dk,dv,pad,packed", SCAN)
def test_scan(gdn, lens, nk, nv, dk, dv, pad, packed, steps, rate):
    s = ssm(lens, nk, nv, dk, dv, pad, steps=steps, rate=rate)
    want = ssm_want(s, lens)
    rows = sum(lens)
    out = torch.full((rows + 2, nv * dv + 8), 7.0, dtype=torch.bfloat16, device=DEV)
    state = s["state"].clone()
    gdn.ssm_scan(s["q"], s["k"], s["v"], s["dt"], s["a"], state, out[1:-1, :nv * dv], **s["args"], **batch(lens, packed))
    gdn.check()
    check_scan(out[1:-1, :nv * dv].reshape(rows, -1), state, want, rows)
    assert (out[0] == 7).all() and (out[-1] == 7).all() and (out[:, nv * dv:] == 7).all()
    for i, n in enumerate(lens):
        if n == 0:
            assert torch.equal(state[i], s["state"][i])


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("softplus,skip", [(True, False), (False, True), (False, False)])
def test_scan_forms_of_the_step(gdn, dt, softplus, skip):
    lens = [150, 64]
    s = ssm(lens, 1, 2, 128, 64, dt=dt, softplus=softplus, skip=skip, seed=5)
    if not softplus:
        s["args"]["dt_bias"] = None
    want = ssm_want(s, lens)
    out, state = torch.empty(sum(lens), 128, dtype=torch.bfloat16, device=DEV), s["state"].clone()
    gdn.ssm_scan(s["q"], s["k"], s["v"], s["dt"], s["a"], state, out, **s["args"], **batch(lens, True))
    gdn.check()
    check_scan(out, state, want, sum(lens))


def test_scan_nothing_from_behind_a_sequence(gdn):
    """Rows behind a sequence's last token, NaN and infinities among them, reach neither it nor its state; rows behind the last
    sequence are left as they are."""
    for steps, rate in ((0.05, 8.0), (3.0, 30.0)):
        lens = [200, 77]
        s = ssm(lens, 1, 2, 128, 64, seed=7, steps=steps, rate=rate)
        want = ssm_want(s, lens)
        bad = {n: torch.cat([s[n], torch.full((200, s[n].shape[1]), float("nan"), dtype=s[n].dtype, device=DEV)]) for n in ("q", "k", "v", "dt")}
        for n in ("q", "k", "v", "dt"):
            bad[n][-50:] = float("inf")
        out, state = torch.full((477, 128), 7.0, dtype=torch.bfloat16, device=DEV), s["state"].clone()
        gdn.ssm_scan(bad["q"], bad["k"], bad["v"], bad["dt"], s["a"], state, out, **s["args"], **batch(lens, True))
        gdn.check()
        check_scan(out[:277], state, want, 277)
        assert (out[277:] == 7).all()


DECODE = [(1, 1, 1, 64, 64, 0), (3, 1, 24, 128, 64, 8), (5, 2, 6, 64, 128, 0), (17, 4, 4, 128, 128, 16)]


@pytest.mark.parametrize("B,nk,nv,dk,dv,pad", DECODE)
def test_decode(gdn, B, nk, nv, dk, dv, pad):
    s = ssm([1] * B, nk, nv, dk, dv, pad, steps=0.5)
    o, S, mags, M = ssm_want(s, [1] * B)
    out, state = torch.empty(B, nv * dv, dtype=torch.bfloat16, device=DEV), s["state"].clone()
    gdn.ssm_decode(s["q"], s["k"], s["v"], s["dt"], s["a"], state, out, **s["args"])
    gdn.check()
    # the exponent is off by a few fp32 steps of itself (at most 4 here), the rest are single roundings
    near(state, S, 64 * ref.U * M, "state")
    near(out.view(o.shape), o, (64 + dk) * ref.U * mags + ref.half(torch.bfloat16) * o.abs() + 1e-30, "out")


def test_decode_goes_on_where_the_scan_stops(gdn):
    """A prompt in one call, in two, and its last tokens one by one: the same states and outputs within their bounds."""
    T, cut = 150, 147
    s = ssm([T], 2, 4, 128, 64, seed=11)
    want = ssm_want(s, [T])
    out, state = torch.empty(T, 256, dtype=torch.bfloat16, device=DEV), s["state"].clone()
    part = lambda a, b: [s[n][a:b] for n in ("q", "k", "v", "dt")]  # noqa: E731
    gdn.ssm_scan(*part(0, 100), s["a"], state, out[:100], B=1, T=100, **s["args"])
    gdn.ssm_scan(*part(100, cut), s["a"], state, out[100:cut], B=1, T=cut - 100, **s["args"])
    for t in range(cut, T):
        gdn.ssm_decode(*part(t, t + 1), s["a"], state, out[t:t + 1], **s["args"])
    gdn.check()
    check_scan(out, state, want, T)


def test_state_tables(gdn):
    lens = [70, 3]
    s = ssm(lens, 1, 2, 128, 64, seed=13)
    out, state = torch.empty(2, sum(lens), 128, dtype=torch.bfloat16, device=DEV), s["state"].clone()
    gdn.ssm_scan(s["q"], s["k"], s["v"], s["dt"], s["a"], state, out[0], **s["args"], **batch(lens, True))
    apart = [s["state"][i].clone() for i in (1, 0)]
    table = torch.tensor([apart[1].data_ptr(), apart[0].data_ptr()], device=DEV)
    gdn.ssm_scan(s["q"], s["k"], s["v"], s["dt"], s["a"], table, out[1], state_is_table=True, **s["args"], **batch(lens, True))
    assert torch.equal(out[0], out[1]) and torch.equal(apart[1], state[0]) and torch.equal(apart[0], state[1])
    rows = dict(q=s["q"][:2], k=s["k"][:2], v=s["v"][:2], dt=s["dt"][:2])
    gdn.ssm_decode(*rows.values(), s["a"], state, out[0][:2], **s["args"])
    gdn.ssm_decode(*rows.values(), s["a"], table, out[1][:2], state_is_table=True, **s["args"])
    assert torch.equal(out[0][:2], out[1][:2]) and torch.equal(apart[1], state[0])
    for lens in ([1, 1], [400, 3]):
        c = make_conv(lens, 128, 4, torch.bfloat16)
        kept, apart = c["h0"].clone(), [c["h0"][i].clone() for i in range(2)]
        a, b = torch.empty_like(c["x"]), torch.empty_like(c["x"])
        gdn.causal_conv(c["x"], c["w"], a, bias=c["b"], state=kept, **batch(lens, lens[0] != lens[1]))
        gdn.causal_conv(c["x"], c["w"], b, bias=c["b"], state=torch.tensor([t.data_ptr() for t in apart], device=DEV), state_is_table=True,
                        **batch(lens, lens[0] != lens[1]))
        assert torch.equal(a, b) and torch.equal(kept, torch.stack(apart))
    gdn.check()


NORM = [  # rows, groups, dim, type, padding
    (1, 1, 8, "bf16", 0), (3, 5, 16, "fp32", 8), (37, 3, 24, "fp16", 0), (50, 2, 64, "bf16", 8), (129, 32, 128, "bf16", 0),
    (9, 7, 120, "fp32", 0), (65, 2, 256, "fp16", 16), (33, 1, 264, "bf16", 0), (20, 2, 1000, "fp32", 0), (301, 1, 1024, "bf16", 0),
    (17, 1, 1032, "fp16", 8), (700, 1, 4096, "bf16", 0), (5, 1, 4104, "fp32", 0), (11, 2, 8192, "bf16", 0), (3, 1, 8192, "fp32", 0),
]
FORMS = [("layer", None), ("rms", None), ("layer", "after"), ("rms", "after"), ("layer", "before"), ("rms", "before")]


def make_norm(rows, groups, dim, dtype, pad, kind, gate, plain=False, seed=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    w = groups * dim
    return dict(x=wide(gen, rows, w, dtype, pad) + rand(gen, rows, 1, dtype=dtype), gate=wide(gen, rows, w, dtype, pad) if gate else None,
                weight=None if plain else 1 + 0.1 * rand(gen, dim), bias=None if plain else 0.1 * rand(gen, dim), dout=wide(gen, rows, w, dtype, pad),
                form=dict(dim=dim, gate_first=gate == "before", rms=kind == "rms", eps=1e-5))


def grouped(t, dim):
    return None if t is None else t.double().unflatten(-1, (-1, dim)) if t.dim() > 1 else t.double()


@pytest.mark.parametrize("kind,gate", FORMS)
@pytest.mark.parametrize("rows,groups,dim,type,pad", NORM)
def test_norm_and_backward(gdn, rows, groups, dim, type, pad, kind, gate):
    dtype = TYPES[type]
    c = make_norm(rows, groups, dim, dtype, pad, kind, gate, plain=(rows + dim) % 3 == 0)
    leaf = {n: grouped(c[n], dim).detach().clone().requires_grad_(True) for n in ("x", "gate", "weight", "bias") if c[n] is not None}
    f = c["form"]
    want = ref.norm(leaf["x"], leaf.get("weight"), leaf.get("bias"), leaf.get("gate"), f["gate_first"], f["rms"], f["eps"])
    dout = grouped(c["dout"], dim)
    (want * dout).sum().backward()
    out = torch.full((rows + 2, groups * dim + 8), 7.0, dtype=dtype, device=DEV)
    gdn.layer_norm(c["x"], out[1:-1, :-8], weight=c["weight"], bias=c["bias"], gate=c["gate"], **f)
    dx, dgate = torch.full_like(c["dout"], 7).contiguous(), torch.full_like(c["dout"], 7).contiguous() if gate else None
    dw, db = torch.full((dim,), 7.0, device=DEV), torch.full((dim,), 7.0, device=DEV)
    gdn.layer_norm_backward(c["x"], c["dout"], dx, dw, db, weight=c["weight"], bias=c["bias"], gate=c["gate"], dgate=dgate, **f)
    gdn.check()
    with torch.no_grad():
        z = leaf.get("gate")
        g = (z * torch.sigmoid(z)).abs() if z is not None else torch.ones_like(leaf["x"])
        zs = z.abs() + 8 if z is not None else 0.0
        u = leaf["x"] * (z * torch.sigmoid(z) if f["gate_first"] else 1.0)
        m = 0.0 if f["rms"] else u.mean(-1, keepdim=True)
        r = 1 / torch.sqrt(((u - m) ** 2).mean(-1, keepdim=True) + f["eps"])
        h = (u - m) * r
        w = leaf["weight"].abs() if "weight" in leaf else torch.ones(dim, device=DEV, dtype=torch.float64)
        b = leaf["bias"].abs() if "bias" in leaf else 0.0
        # h: u and its mean within 16 + |z| / 2 fp32 steps of the group's size (sums of 32 a thread, then by halves), r within 24 of its own
        size = u.abs() + u.abs().mean(-1, keepdim=True)
        dh = (32 + 2 * zs) * ref.U * (size * r + h.abs())
        after = g if z is not None and not f["gate_first"] else 1.0
        y = (h.abs() * w + b) * after
        near(out[1:-1, :-8].unflatten(1, (groups, dim)), want, dh * w * after + (8 + 2 * zs) * ref.U * y + ref.half(dtype) * want.abs() + ref.least(dtype), "out")
        assert (out[0] == 7).all() and (out[-1] == 7).all() and (out[:, -8:] == 7).all()
        # backward: t = dout w (times silu(z)), du = r (t - mean t - h mean(t h))
        t = dout.abs() * w * after
        mean_t, mean_th = t.mean(-1, keepdim=True), (t * h.abs()).mean(-1, keepdim=True)
        du = r * (t + (0 if f["rms"] else mean_t) + h.abs() * mean_th)
        off = (96 + 8 * zs) * ref.U * du + r * (dh * mean_th + h.abs() * (t * dh).mean(-1, keepdim=True))
        x = leaf["x"]
        slope = 1.1
        if f["gate_first"]:
            near(dx.unflatten(1, (groups, dim)), x.grad, off * g + 8 * ref.U * du * g + ref.half(dtype) * x.grad.abs() + ref.least(dtype), "dx")
            near(dgate.unflatten(1, (groups, dim)), z.grad, (off + (16 + 4 * zs) * ref.U * du) * x.abs() * slope + ref.half(dtype) * z.grad.abs() + ref.least(dtype),
                 "dgate")
        else:
            near(dx.unflatten(1, (groups, dim)), x.grad, off + ref.half(dtype) * x.grad.abs() + ref.least(dtype), "dx")
            if z is not None:
                near(dgate.unflatten(1, (groups, dim)), z.grad,
                     slope * dout.abs() * (dh * w + (16 + 4 * zs) * ref.U * (h.abs() * w + b)) + ref.half(dtype) * z.grad.abs() + ref.least(dtype), "dgate")
        g_out = dout * (z * torch.sigmoid(z) if z is not None and not f["gate_first"] else 1.0)
        n = rows * groups
        want_w, want_b = (g_out * h).sum((0, 1)), g_out.sum((0, 1))
        near(dw, want_w, (g_out.abs() * dh).sum((0, 1)) + (n + 16) * ref.U * (g_out * h).abs().sum((0, 1)) + 8 * ref.U * ((zs + 1) * (g_out * h).abs()).sum((0, 1)) + 1e-30, "dweight")
        near(db, want_b, (n + 16) * ref.U * g_out.abs().sum((0, 1)) + 8 * ref.U * ((zs + 1) * g_out.abs()).sum((0, 1)) + 1e-30, "dbias")


def test_norm_in_place(gdn):
    c = make_norm(40, 2, 128, torch.bfloat16, 0, "rms", "after")
    f = c["form"]
    out, x, z = torch.empty_like(c["x"]), c["x"].clone(), c["gate"].clone()
    gdn.layer_norm(c["x"], out, weight=c["weight"], gate=c["gate"], **f)
    gdn.layer_norm(x, x, weight=c["weight"], gate=c["gate"], **f)
    gdn.layer_norm(c["x"], z, weight=c["weight"], gate=z, **f)
    assert torch.equal(out, x) and torch.equal(out, z)
    dx, dz, g, z = torch.empty_like(x), torch.empty_like(x), c["dout"].clone(), c["gate"].clone()
    gdn.layer_norm_backward(c["x"], c["dout"], dx, weight=c["weight"], gate=c["gate"], dgate=dz, **f)
    gdn.layer_norm_backward(c["x"], g, g, weight=c["weight"], gate=z, dgate=z, **f)
    gdn.check()
    assert torch.equal(dx, g) and torch.equal(dz, z)


def test_norm_backward_against_differences(gdn):
    """The gradients as slopes of the forward itself, in fp32."""
    for kind, gate in FORMS:
        c = make_norm(6, 2, 40, torch.float32, 0, kind, gate, seed=4)
        f = c["form"]
        dx, dz = torch.empty_like(c["x"]), torch.empty_like(c["x"]) if gate else None
        dw, db = torch.empty_like(c["weight"]), torch.empty_like(c["bias"])
        gdn.layer_norm_backward(c["x"], c["dout"], dx, dw, db, weight=c["weight"], bias=c["bias"], gate=c["gate"], dgate=dz, **f)

        def loss(**kw):
            out = torch.empty_like(c["x"])
            a = dict(x=c["x"], weight=c["weight"], bias=c["bias"], gate=c["gate"])
            a.update(kw)
            gdn.layer_norm(a.pop("x"), out, **a, **f)
            return float((out.double() * c["dout"].double()).sum())

        gen, step, size = torch.Generator(device=DEV).manual_seed(8), 2.0 ** -8, float(c["dout"].abs().sum())
        for name, grad in (("x", dx), ("weight", dw), ("bias", db)) + ((("gate", dz),) if gate else ()):
            along = torch.randn(grad.shape, generator=gen, device=DEV)
            up, down = (loss(**{name: c[name] + sign * step * along}) for sign in (1, -1))
            slope, want = (up - down) / (2 * step), float((grad.double() * along.double()).sum())
            # third derivatives: a few times the output's size x |along|^3 / deviation^3 (about 1 here; smaller where the gate comes first)
            assert abs(slope - want) <= 64 * step ** 2 * size + size * 2 ** -20 / step, (kind, gate, name)


def test_same_inputs_same_bits(gdn):
    """The sums of the weights' gradients have a fixed order, whatever the workspace."""
    c = make_conv([300, 41, 0, 7], 264, 4, torch.bfloat16)
    got = []
    for ws in (None, torch.full((gdn.causal_conv_backward_workspace_bytes(348, 264, 4),), 255, dtype=torch.uint8, device=DEV)):
        dx, dw, db = torch.empty_like(c["x"]), torch.empty_like(c["w"]), torch.empty_like(c["b"])
        gdn.causal_conv_backward(c["x"], c["w"], c["dout"], dx, dw, db, bias=c["b"], h0=c["h0"], workspace=ws, **batch([300, 41, 0, 7], True))
        got.append((dx, dw, db))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    n = make_norm(501, 1, 2048, torch.bfloat16, 0, "layer", None)
    got = []
    for ws in (None, torch.full((gdn.layer_norm_backward_workspace_bytes(501, 1, 2048),), 255, dtype=torch.uint8, device=DEV)):
        dx, dw, db = torch.empty_like(n["x"]), torch.empty_like(n["weight"]), torch.empty_like(n["weight"])
        gdn.layer_norm_backward(n["x"], n["dout"], dx, dw, db, weight=n["weight"], bias=n["bias"], workspace=ws, **n["form"])
        got.append((dx, dw, db))
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_no_rows(gdn):
    e = lambda *s, dtype=torch.bfloat16: torch.empty(*s, dtype=dtype, device=DEV)  # noqa: E731
    w, b, dw, db = torch.ones(64, 4, device=DEV), torch.ones(64, device=DEV), torch.full((64, 4), 7.0, device=DEV), torch.full((64,), 7.0, device=DEV)
    gdn.causal_conv(e(0, 64), w, e(0, 64), bias=b, B=3, T=0)
    dh0, dST = e(2, 3, 64), rand(torch.Generator(device=DEV).manual_seed(0), 2, 3, 64, dtype=torch.bfloat16)
    gdn.causal_conv_backward(e(0, 64), w, e(0, 64), e(0, 64), dw, db, h0=e(2, 3, 64), dST=dST, dh0=dh0, B=2, T=0)
    assert (dw == 0).all() and (db == 0).all() and torch.equal(dh0, dST)
    gdn.layer_norm(e(0, 128), e(0, 128), dim=64)
    db = torch.full((64,), 7.0, device=DEV)
    gdn.layer_norm_backward(e(0, 128), e(0, 128), e(0, 128), db, None, dim=64)
    assert (db == 0).all()
    f32 = dict(dtype=torch.float32)
    gdn.ssm_scan(e(0, 128), e(0, 128), e(0, 128), e(0, 2, **f32), e(2, **f32), e(0, 2, 128, 64, **f32), e(0, 128), nk=1, nv=2, dv=64, B=0, T=5)
    gdn.ssm_decode(e(0, 128), e(0, 128), e(0, 128), e(0, 2, **f32), e(2, **f32), e(0, 2, 128, 64, **f32), e(0, 128), nk=1, nv=2, dv=64)
    gdn.check()


@pytest.mark.parametrize("cu", [[0, 50, 40, 90], [5, 40, 60, 90], [0, 200, 60, 90], [-4, 40, 60, 90], [0, 40, 60, 200], [0, 2 ** 31 - 1, 60, 90]])
def test_bad_offsets_are_reported(gdn, cu):
    """Sequences whose offsets fall, or leave the rows, are skipped and reported; nothing outside the outputs is touched."""
    bad = torch.tensor(cu, dtype=torch.int32, device=DEV)
    ok = [0 <= cu[i] <= cu[i + 1] <= 90 for i in range(3)]
    s = ssm([30] * 3, 1, 2, 128, 64)
    c = make_conv([30] * 3, 64, 4, torch.bfloat16)

    def calls():
        out, state = torch.full((90, 128), 7.0, dtype=torch.bfloat16, device=DEV), s["state"].clone()
        yield lambda: gdn.ssm_scan(s["q"], s["k"], s["v"], s["dt"], s["a"], state, out, cu_seqlens=bad, **s["args"])
        assert all(torch.equal(state[i], s["state"][i]) for i in range(3) if not ok[i])
        y, kept = torch.full((90, 64), 7.0, dtype=torch.bfloat16, device=DEV), c["h0"].clone()
        yield lambda: gdn.causal_conv(c["x"], c["w"], y, bias=c["b"], state=kept, cu_seqlens=bad)
        assert all(torch.equal(kept[i], c["h0"][i]) for i in range(3) if not ok[i])
        dx, dw = torch.empty_like(c["x"]), torch.empty_like(c["w"])
        yield lambda: gdn.causal_conv_backward(c["x"], c["w"], c["dout"], dx, dw, bias=c["b"], h0=c["h0"], dh0=torch.empty_like(c["h0"]), cu_seqlens=bad)

    for call in calls():
        call()
        with pytest.raises(gdn.GdnError) as e:
            gdn.check()
        assert e.value.code == gdn.GDN_ERR_DEVICE_STATUS
        gdn.check()


def test_other_stream_and_graph(gdn):
    """On another stream, and captured with its own workspace and replayed on other inputs."""
    lens = [150, 260]
    s, c, n = ssm(lens, 1, 2, 128, 64, seed=21), make_conv(lens, 128, 4, torch.bfloat16, seed=21), make_norm(410, 2, 64, torch.bfloat16, 0, "rms", "after", seed=21)
    b = batch(lens, True)
    ws = torch.empty(max(gdn.ssm_scan_workspace_bytes(2, 410, 1, 2, True, dv=64), gdn.causal_conv_backward_workspace_bytes(410, 128, 4),
                         gdn.layer_norm_backward_workspace_bytes(410, 2, 64), 1), dtype=torch.uint8, device=DEV)
    outs = [torch.empty(410, 128, dtype=torch.bfloat16, device=DEV) for _ in range(5)]
    state, kept, dw, dnw = s["state"].clone(), c["h0"].clone(), torch.empty_like(c["w"]), torch.empty_like(n["weight"])

    def run():
        state.copy_(s["state"])
        kept.copy_(c["h0"])
        gdn.causal_conv(c["x"], c["w"], outs[0], bias=c["b"], state=kept, **b)
        gdn.causal_conv_backward(c["x"], c["w"], c["dout"], outs[1], dw, bias=c["b"], h0=c["h0"], workspace=ws, **b)
        gdn.ssm_scan(s["q"], s["k"], s["v"], s["dt"], s["a"], state, outs[2], workspace=ws, **s["args"], **b)
        gdn.layer_norm(n["x"], outs[3], weight=n["weight"], gate=n["gate"], **n["form"])
        gdn.layer_norm_backward(n["x"], n["dout"], outs[4], dnw, weight=n["weight"], gate=n["gate"], dgate=torch.empty_like(n["x"]), workspace=ws, **n["form"])
        return [t.clone() for t in outs + [state, kept, dw, dnw]]

    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = run()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(x, y) for x, y in zip(want, again))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for t in (s["v"], c["x"], n["x"]):
        t.neg_()
    graph.replay()
    other = [t.clone() for t in got]
    want = run()
    assert all(torch.equal(x, y) for x, y in zip(want, other))
    gdn.check()


def test_layer_of_them(gdn):
    """As a linear-attention layer runs them: convolution, its slices into the delta rule and into the scan, the gated norm; a prompt
    and then single tokens, against the whole sequence at once."""
    nk, nv, T, cut = 1, 2, 90, 87
    gen = torch.Generator(device=DEV).manual_seed(33)
    width = 2 * nk * 128 + nv * 128
    x, w = rand(gen, T, width, dtype=torch.bfloat16), rand(gen, width, 4, scale=0.5)
    gate, dt, a = rand(gen, T, nv * 128, dtype=torch.bfloat16), rand(gen, T, nv), -torch.rand(nv, generator=gen, device=DEV)
    g, beta = -torch.rand(T, nv, generator=gen, device=DEV), torch.rand(T, nv, generator=gen, device=DEV)
    weight = 1 + 0.1 * rand(gen, 128)

    def run(cuts):
        conv_state = torch.zeros(1, 3, width, dtype=torch.bfloat16, device=DEV)
        S = [torch.zeros(1, nv, 128, 128, device=DEV) for _ in range(2)]
        mixed, y, o = torch.empty_like(x), [torch.empty_like(gate) for _ in range(2)], [torch.empty_like(gate) for _ in range(2)]
        for i, j in zip(cuts[:-1], cuts[1:]):
            gdn.causal_conv(x[i:j], w, mixed[i:j], state=conv_state, B=1, T=j - i)
            q, k, v = mixed[i:j, :128], mixed[i:j, 128:256], mixed[i:j, 256:]
            if j - i > 1:
                gdn.prefill(q, k, v, g[i:j], beta[i:j], S[0], y[0][i:j], nk=nk, nv=nv, B=1, T=j - i, qk_l2norm=True)
                gdn.ssm_scan(q, k, v, dt[i:j], a, S[1], y[1][i:j], nk=nk, nv=nv, B=1, T=j - i)
            else:
                gdn.decode(q, k, v, g[i:j], beta[i:j], S[0], y[0][i:j], nk=nk, nv=nv, qk_l2norm=True)
                gdn.ssm_decode(q, k, v, dt[i:j], a, S[1], y[1][i:j], nk=nk, nv=nv)
            for u in range(2):
                gdn.layer_norm(y[u][i:j], o[u][i:j], dim=128, weight=weight, gate=gate[i:j], rms=True)
        gdn.check()
        return mixed, conv_state, y, S, o

    one, parts = run([0, T]), run([0, 50, cut] + list(range(cut + 1, T + 1)))
    assert torch.equal(one[0], parts[0]) and torch.equal(one[1], parts[1])
    for u, bar in ((0, 1e-2), (1, 5e-3)):
        for p, q in ((one[2][u], parts[2][u]), (one[4][u], parts[4][u])):
            assert float((p.double() - q.double()).norm()) <= 2 * bar * float(p.double().norm())
        assert float((one[3][u] - parts[3][u]).norm()) <= 2e-3 * float(one[3][u].norm())


@pytest.mark.parametrize("lens,nk,nv,dk,dv,packed", [
    ([5000], 1, 3, 128, 64, False), ([4100, 4100], 2, 4, 64, 64, False), ([6001], 1, 1, 128, 128, False), ([2500] * 3, 1, 2, 64, 128, False),
    ([7000, 3, 0, 130], 1, 4, 128, 64, True), ([0, 9000], 1, 2, 64, 64, True), ([600] * 32, 1, 2, 64, 64, True), ([40] * 40 + [900], 1, 2, 64, 64, True),
])
def test_scan_in_segments(gdn, lens, nk, nv, dk, dv, packed):
    """Long sequences on few heads, whose segments run side by side, among short ones; more sequences than one warp looks at."""
    for steps, rate in ((0.02, 2.0), (0.5, 8.0)):
        s = ssm(lens, nk, nv, dk, dv, steps=steps, rate=rate, seed=len(lens))
        want = ssm_want(s, lens)
        size = gdn.ssm_scan_workspace_bytes(len(lens), sum(lens) if packed else lens[0], nk, nv, packed, dk=dk, dv=dv)
        got = []
        for ws in (None, torch.full((max(size, 1),), 255, dtype=torch.uint8, device=DEV)):
            out, state = torch.empty(sum(lens), nv * dv, dtype=torch.bfloat16, device=DEV), s["state"].clone()
            gdn.ssm_scan(s["q"], s["k"], s["v"], s["dt"], s["a"], state, out, workspace=ws, **s["args"], **batch(lens, packed))
            got.append((out, state))
        gdn.check()
        assert all(torch.equal(a, b) for a, b in zip(*got))
        check_scan(*got[0], want, sum(lens))


def test_scan_over_decays_of_all_sizes(gdn):
    """Chunks that decay by little and by much in one sequence, heads of both kinds side by side, and tokens that reset the state:
    a step so large that its decay is none in fp32 leaves the tokens before it as exact as the others."""
    lens = [900, 390]
    for dk, dv, nk, nv in ((128, 64, 1, 4), (64, 64, 2, 6), (128, 128, 1, 2)):
        s = ssm(lens, nk, nv, dk, dv, seed=17, steps=0.05, rate=8.0)
        rows = sum(lens)
        gen = torch.Generator(device=DEV).manual_seed(3)
        s["dt"][130:256, ::2] += 5.0
        s["dt"][256:384] += 2.0
        s["dt"][500:640, 1::2] += 8.0
        at = torch.randperm(rows, generator=gen, device=DEV)[:12]
        s["dt"][at] = torch.tensor([30.0, 1e3, 1e5, 1e7, 1e9, 300.0] * 2, device=DEV)[:, None]
        s["v"][at] = (s["v"][at].float() * 1e-3).to(torch.bfloat16)
        z = s["dt"].double() + s["bias"].double()
        s["d"] = torch.logaddexp(z, torch.zeros_like(z))  # softplus without an overflow at any size
        want = ssm_want(s, lens)
        out, state = torch.empty(rows, nv * dv, dtype=torch.bfloat16, device=DEV), s["state"].clone()
        gdn.ssm_scan(s["q"], s["k"], s["v"], s["dt"], s["a"], state, out, **s["args"], **batch(lens, True))
        gdn.check()
        o, S, mags, M = want
        near(out.view(o.shape), o, 2.0 ** -6 * mags + 2.0 ** -8 * o.abs() + 1e-30, "out")
        near(state, S, 2.0 ** -14 * M + 1e-30, "state")


def calls_of_each(gdn, seed, given):
    """A call of every operator, with workspaces of its own (`given`) or the stream's; outputs are the call's. A dense scan in segments
    among them."""
    lens = [150, 0, 260]
    s, c = ssm(lens, 1, 2, 128, 64, seed=seed), make_conv(lens, 128, 4, torch.bfloat16, seed=seed)
    n, m = make_norm(410, 2, 64, torch.bfloat16, 0, "rms", "after", seed=seed), make_norm(300, 1, 1000, torch.float16, 8, "layer", None, seed=seed)
    long = ssm([4000], 1, 2, 64, 64, seed=seed)
    b, one = batch(lens, True), batch([4000], False)
    space = lambda size: torch.empty(max(size, 1), dtype=torch.uint8, device=DEV) if given else None
    sizes = [gdn.causal_conv_backward_workspace_bytes(410, 128, 4), gdn.ssm_scan_workspace_bytes(3, 410, 1, 2, True, dv=64),
             gdn.ssm_scan_workspace_bytes(1, 4000, 1, 2, False, dk=64, dv=64), gdn.layer_norm_backward_workspace_bytes(410, 2, 64),
             gdn.layer_norm_backward_workspace_bytes(300, 1, 1000)]
    assert sizes[2] > 0  # it goes in segments
    ws = [space(x) for x in sizes]
    bf = lambda *shape: torch.empty(*shape, dtype=torch.bfloat16, device=DEV)
    o = [bf(410, 128) for _ in range(5)] + [bf(4000, 128), torch.empty(300, 1000, dtype=torch.float16, device=DEV), bf(410, 128)]
    states = [s["state"].clone(), long["state"].clone(), s["state"].clone(), c["h0"].clone()]
    sums = [torch.empty_like(t) for t in (c["w"], c["b"], n["weight"], m["weight"], m["weight"])] + [torch.empty_like(c["h0"])]

    def run():
        for t, f in zip(states, (s["state"], long["state"], s["state"], c["h0"])):
            t.copy_(f)
        gdn.causal_conv_backward(c["x"], c["w"], c["dout"], o[1], sums[0], sums[1], bias=c["b"], h0=c["h0"], dh0=sums[5], workspace=ws[0], **b)
        gdn.causal_conv(c["x"], c["w"], o[0], bias=c["b"], state=states[3], **b)
        gdn.ssm_scan(s["q"], s["k"], s["v"], s["dt"], s["a"], states[0], o[2], workspace=ws[1], **s["args"], **b)
        gdn.ssm_scan(long["q"], long["k"], long["v"], long["dt"], long["a"], states[1], o[5], workspace=ws[2], **long["args"], **one)
        gdn.ssm_decode(s["q"][:3], s["k"][:3], s["v"][:3], s["dt"][:3], s["a"], states[2], o[3][:3], **s["args"])
        gdn.layer_norm_backward(n["x"], n["dout"], o[4], sums[2], weight=n["weight"], gate=n["gate"], dgate=o[7], workspace=ws[3], **n["form"])
        gdn.layer_norm(n["x"], o[3], weight=n["weight"], gate=n["gate"], **n["form"])
        gdn.layer_norm_backward(m["x"], m["dout"], o[6], sums[3], sums[4], weight=m["weight"], workspace=ws[4], **m["form"])

    return run, lambda: [t.clone() for t in o + states + sums]


@pytest.mark.parametrize("given", [True, False])
def test_calls_that_overlap(gdn, given):
    """Two runs of every operator at once, on two streams, as calls and as graphs, each against its own run alone."""
    runs = [calls_of_each(gdn, seed, given) for seed in (41, 42)]
    want = []
    for run, got in runs:
        run()
        torch.cuda.synchronize()
        want.append(got())
    sides = [torch.cuda.Stream() for _ in runs]

    def check():
        torch.cuda.synchronize()
        for w, (_, got) in zip(want, runs):
            assert all(torch.equal(x, y) for x, y in zip(w, got()))

    for _ in range(3):
        for side, (run, _) in zip(sides, runs):
            with torch.cuda.stream(side):
                run()
    check()
    graphs = []
    for side, (run, _) in zip(sides, runs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=side):
            run()
    for _ in range(3):
        for side, graph in zip(sides, graphs):
            with torch.cuda.stream(side):
                graph.replay()
    check()
    for run, _ in runs:  # and calls beside a graph
        run()
    check()
    gdn.check()


def test_offsets_past_32_bits(gdn):
    """Rows that lie 2^29 elements apart, so that the last ones' offsets pass 32 bits, against the same rows packed."""
    rows, far = 5, 1 << 29
    s, c = ssm([2, 3], 1, 2, 128, 64, seed=51), make_conv([2, 3], 128, 4, torch.bfloat16, seed=51)
    n = make_norm(rows, 2, 64, torch.bfloat16, 0, "rms", "after", seed=51)
    b = batch([2, 3], True)
    space = torch.empty(rows * far, dtype=torch.bfloat16, device=DEV)
    used = [0]

    def apart(t):  # the same rows, far from one another
        v = space.as_strided((rows, t.shape[1]), (far, 1), used[0])
        used[0] += 256
        return v.copy_(t)

    outs = []
    for wide_apart in (False, True):
        put = apart if wide_apart else lambda t: t.clone()
        bf = lambda w=128: put(torch.zeros(rows, w, dtype=torch.bfloat16, device=DEV))
        o = [bf() for _ in range(7)]
        states = [c["h0"].clone(), s["state"].clone(), s["state"][:1].expand(rows, -1, -1, -1).contiguous()]
        sums = [torch.empty_like(c["w"]), torch.empty_like(n["weight"])]
        x, dout, q, k, v, z, g = (put(t) for t in (c["x"], c["dout"], s["q"], s["k"], s["v"], n["gate"], n["x"]))
        gdn.causal_conv(x, c["w"], o[0], bias=c["b"], state=states[0], **b)
        gdn.causal_conv_backward(x, c["w"], dout, o[1], sums[0], bias=c["b"], h0=c["h0"], **b)
        gdn.ssm_scan(q, k, v, s["dt"], s["a"], states[1], o[2], **s["args"], **b)
        gdn.ssm_decode(q, k, v, s["dt"], s["a"], states[2], o[3], **s["args"])
        gdn.layer_norm(g, o[4], weight=n["weight"], gate=z, **n["form"])
        gdn.layer_norm_backward(g, dout, o[5], sums[1], weight=n["weight"], gate=z, dgate=o[6], **n["form"])
        gdn.check()
        outs.append([t.clone() for t in o + states + sums])
    assert all(torch.equal(x, y) for x, y in zip(*outs))


def test_states_past_32_bits(gdn):
    """A step of so many heads that the last states' offsets pass 32 bits, against those sequences alone."""
    B, nv = 1100, 128
    gen = torch.Generator(device=DEV).manual_seed(7)
    state = torch.empty(B, nv, 128, 128, device=DEV)
    state[-2:] = rand(gen, 2, nv, 128, 128)
    state[:-2] = 0
    bf = torch.bfloat16
    q, k, v = rand(gen, B, 128, dtype=bf), rand(gen, B, 128, dtype=bf), rand(gen, B, nv * 128, dtype=bf)
    dt, a = rand(gen, B, nv), -torch.rand(nv, generator=gen, device=DEV)
    assert state.numel() > 2 ** 31
    few, out, one = state[-2:].clone(), torch.empty_like(v), torch.empty_like(v[-2:])
    gdn.ssm_decode(q, k, v, dt, a, state, out, nk=1, nv=nv)
    gdn.ssm_decode(q[-2:], k[-2:], v[-2:], dt[-2:], a, few, one, nk=1, nv=nv)
    gdn.check()
    assert torch.equal(state[-2:], few) and torch.equal(out[-2:], one)
    d = torch.nn.functional.softplus(dt[0].double())
    # the first sequence from nothing: k (d v)^T, d off by 4 steps of fp32, the products by one each
    want = k[0].double()[None, :, None] * (d[:, None] * v[0].double().view(nv, 128))[:, None, :]
    near(state[0], want, 2.0 ** -20 * want.abs() + 1e-30, "state")
