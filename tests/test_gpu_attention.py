"""GPU tests of the softmax-attention operators (head norm with rotation and its backward, paged append, tree
attention) against their plain 64-bit forms, with error bounds that follow from the kernels' roundings."""
import math

import pytest

torch = pytest.importorskip("torch")

from tests import attention_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_delta_rule_17_gb300 import build

    build.build()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype=BF):
    return torch.randn(shape, generator=g).to(dtype)


def padded(x, pad):
    """x [rows, ...] on the GPU in rows that are `pad` elements longer."""
    rows, inner = x.shape[0], x[0].numel() if x.shape[0] else math.prod(x.shape[1:])
    wide = torch.full((rows, inner + pad), float("nan"), dtype=x.dtype, device="cuda")
    view = wide[:, :inner]
    view.copy_(x.reshape(rows, inner))
    return view


# ---- norm and rotation -----------------------------------------------------------------


def _norm_case(seed, rows, nq, nkv, d, rot, dtype, interleaved, weights=True, pad=0, table=97):
    g = gen(seed)
    c = dict(rows=rows, nq=nq, nkv=nkv, d=d, dtype=dtype, inter=interleaved, eps=1e-6)
    c["q"], c["k"] = randn(g, rows, nq, d, dtype=dtype), randn(g, rows, nkv, d, dtype=dtype)
    c["gq"], c["gk"] = randn(g, rows, nq, d, dtype=dtype), randn(g, rows, nkv, d, dtype=dtype)
    c["qw"], c["kw"] = (1 + 0.2 * torch.randn(d, generator=g), 1 + 0.2 * torch.randn(d, generator=g)) if weights else (None, None)
    c["cos"], c["sin"] = ref.rope_tables(table, rot) if rot else (None, None)
    c["pos"] = torch.randint(0, table, (rows,), generator=g, dtype=torch.int32)
    c["pad"] = pad
    return c


def _cuda(x):
    return None if x is None else x.cuda()


NORM_CASES = [
    dict(rows=1, nq=16, nkv=2, d=128, rot=128, dtype=BF, interleaved=False),
    dict(rows=37, nq=5, nkv=1, d=128, rot=128, dtype=BF, interleaved=True),
    dict(rows=130, nq=9, nkv=3, d=64, rot=64, dtype=HF, interleaved=False),
    dict(rows=33, nq=17, nkv=8, d=64, rot=16, dtype=BF, interleaved=False),
    dict(rows=64, nq=3, nkv=2, d=128, rot=48, dtype=F32, interleaved=True),
    dict(rows=19, nq=8, nkv=8, d=128, rot=48, dtype=HF, interleaved=False, pad=24),
    dict(rows=1100, nq=12, nkv=4, d=128, rot=128, dtype=F32, interleaved=False, pad=8),
    dict(rows=50, nq=4, nkv=0, d=128, rot=8, dtype=BF, interleaved=False),
    dict(rows=50, nq=0, nkv=4, d=64, rot=8, dtype=BF, interleaved=True),
    dict(rows=21, nq=4, nkv=4, d=128, rot=0, dtype=BF, interleaved=False, weights=False),
]


def _ids(cases):
    return ["-".join(str(v).replace("torch.", "") for v in c.values()) for c in cases]


@pytest.mark.parametrize("case", NORM_CASES, ids=_ids(NORM_CASES))
def test_norm_rope(case):
    import gated_delta_rule_17_gb300 as gdn

    c = _norm_case(11, **case)
    nq, nkv, d, dt = c["nq"], c["nkv"], c["d"], c["dtype"]
    q, k = (padded(c["q"], c["pad"]) if nq else None), (padded(c["k"], c["pad"]) if nkv else None)
    qo = padded(torch.zeros_like(c["q"]), 2 * c["pad"]) if nq else None
    ko = padded(torch.zeros_like(c["k"]), 2 * c["pad"]) if nkv else None
    gdn.head_norm_rope(q, k, c["pos"].cuda(), _cuda(c["cos"]), _cuda(c["sin"]), qo, ko, nq=nq, nkv=nkv, head_dim=d,
                       q_weight=_cuda(c["qw"]), k_weight=_cuda(c["kw"]), eps=c["eps"], interleaved=c["inter"])
    assert gdn.last_launch_count() == 1
    gdn.check()
    at = c["pos"].long()
    cos, sin = (None, None) if c["cos"] is None else (c["cos"][at], c["sin"][at])
    for x, w, y in ((c["q"], c["qw"], qo), (c["k"], c["kw"], ko)):
        if y is None:
            continue
        want = ref.norm_rope(x.double(), w, cos, sin, c["eps"], c["inter"])
        z = ref.norm_rope(x.double(), w, None, None, c["eps"], c["inter"])
        size = z.abs() if cos is None else ref.rotate_sizes(z, 2 * cos.shape[1], c["inter"])
        # fp32: the sum of squares over <= 16 additions in a chain, rsqrt, four products
        bound = ref.ROUNDING[dt] * want.abs() + 32 * ref.FP32 * size + (2.0 ** -25 if dt == HF else 0)
        got = y.cpu().double().view_as(want)
        assert ((got - want).abs() <= bound).all(), float(((got - want).abs() / bound).max())
        if c["pad"]:  # nothing but the rows is written
            assert torch.isnan(y._base[:, x[0].numel():]).all()


def test_norm_rope_in_place_and_empty():
    import gated_delta_rule_17_gb300 as gdn

    c = _norm_case(12, 70, 6, 2, 128, 64, BF, False)
    q, k = c["q"].cuda().flatten(1), c["k"].cuda().flatten(1)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    a = (c["pos"].cuda(), c["cos"].cuda(), c["sin"].cuda())
    kw = dict(nq=6, nkv=2, q_weight=c["qw"].cuda(), k_weight=c["kw"].cuda())
    gdn.head_norm_rope(q, k, *a, qo, ko, **kw)
    gdn.head_norm_rope(q, k, *a, q, k, **kw)
    gdn.check()
    assert torch.equal(q, qo) and torch.equal(k, ko)
    gdn.head_norm_rope(q[:0], k[:0], a[0][:0], *a[1:], qo[:0], ko[:0], **kw)
    assert gdn.last_launch_count() == 0


def test_norm_rope_large_and_zero_rows():
    # a row of zeros stays zero; large fp32 values do not overflow before the mean
    import gated_delta_rule_17_gb300 as gdn

    q = torch.randn(4, 2 * 128, generator=gen(13)).cuda()
    q[1] = 0
    q[2] *= 1e15
    out = torch.empty_like(q)
    gdn.head_norm_rope(q, None, None, None, None, out, None, nq=2, nkv=0)
    gdn.check()
    want = ref.norm_rope(q.cpu().double().view(4, 2, 128), None, None, None, 1e-6, False)
    assert (out[1] == 0).all()
    assert ((out.cpu().double().view_as(want) - want).abs() <= 33 * ref.FP32 * want.abs()).all()


def test_norm_rope_bad_position_is_reported():
    import gated_delta_rule_17_gb300 as gdn

    c = _norm_case(14, 12, 4, 2, 128, 128, BF, False, table=50)
    pos = c["pos"].clone()
    pos[3], pos[7] = 50, -1
    q, k = c["q"].cuda().flatten(1), c["k"].cuda().flatten(1)
    qo, ko = torch.zeros_like(q), torch.zeros_like(k)
    kw = dict(nq=4, nkv=2)
    gdn.head_norm_rope(q, k, pos.cuda(), c["cos"].cuda(), c["sin"].cuda(), qo, ko, **kw)
    with pytest.raises(gdn.GdnError) as e:
        gdn.check()
    assert e.value.code == gdn.GDN_ERR_DEVICE_STATUS and "position" in str(e.value)
    assert (qo[[3, 7]] == 0).all() and (ko[[3, 7]] == 0).all()
    good = [i for i in range(12) if i not in (3, 7)]
    want = ref.norm_rope(c["q"][good].double(), None, c["cos"][pos[good].long()], c["sin"][pos[good].long()], 1e-6, False)
    assert torch.allclose(qo[good].cpu().double().view_as(want), want, rtol=2 ** -7, atol=1e-6)
    gdn.head_norm_rope(q, k, c["pos"].cuda(), c["cos"].cuda(), c["sin"].cuda(), qo, ko, **kw)
    gdn.check()


@pytest.mark.parametrize("case", NORM_CASES, ids=_ids(NORM_CASES))
def test_norm_rope_backward(case):
    import gated_delta_rule_17_gb300 as gdn

    c = _norm_case(15, **case)
    nq, nkv, d, dt, rows = c["nq"], c["nkv"], c["d"], c["dtype"], c["rows"]

    def side(x, g, heads):
        return (padded(x, c["pad"]), padded(g, 2 * c["pad"]), padded(torch.zeros_like(x), 3 * c["pad"])) if heads else (None,) * 3

    q, gq, dq = side(c["q"], c["gq"], nq)
    k, gk, dk = side(c["k"], c["gk"], nkv)
    dqw = torch.full((d,), float("nan"), device="cuda")
    dkw = torch.full((d,), float("nan"), device="cuda")
    args = (q, k, c["pos"].cuda(), _cuda(c["cos"]), _cuda(c["sin"]), gq, gk, dq, dk)
    kw = dict(nq=nq, nkv=nkv, head_dim=d, q_weight=_cuda(c["qw"]), k_weight=_cuda(c["kw"]), eps=c["eps"], interleaved=c["inter"])
    gdn.head_norm_rope_backward(*args, dqw, dkw, **kw)
    assert gdn.last_launch_count() == 2
    gdn.check()
    at = c["pos"].long()
    cos, sin = (None, None) if c["cos"] is None else (c["cos"][at], c["sin"][at])
    for x, g, w, dx, dw in ((c["q"], c["gq"], c["qw"], dq, dqw), (c["k"], c["gk"], c["kw"], dk, dkw)):
        if dx is None:
            assert (dw == 0).all()
            continue
        want, wsum, wsize, size = ref.norm_rope_backward(x.double(), g.double(), w, cos, sin, c["eps"], c["inter"])
        # fp32: two row sums (<= 16 additions in a chain), rsqrt, about ten products and sums
        bound = ref.ROUNDING[dt] * want.abs() + 64 * ref.FP32 * size + (2.0 ** -25 if dt == HF else 0)
        got = dx.cpu().double().view_as(want)
        assert ((got - want).abs() <= bound).all(), float(((got - want).abs() / bound).max())
        # sums over the rows: no chain is longer than the rows and heads themselves (and 16 of a term)
        wbound = (16 + rows * x.shape[1]) * ref.FP32 * wsize + 1e-30
        wgot = dw.cpu().double()
        assert ((wgot - wsum).abs() <= wbound).all(), float(((wgot - wsum).abs() / wbound).max())
    # the same inputs give the same bits; without weight gradients one launch; with a workspace
    again, again_k = torch.empty_like(dqw), torch.empty_like(dkw)
    ws = torch.empty(gdn.head_norm_rope_backward_workspace_bytes(rows, nq, nkv, d), dtype=torch.uint8, device="cuda")
    gdn.head_norm_rope_backward(*args, again, again_k, workspace=ws, **kw)
    assert torch.equal(again, dqw) and torch.equal(again_k, dkw)
    gdn.head_norm_rope_backward(*args, **kw)
    assert gdn.last_launch_count() == 1
    gdn.check()


@pytest.mark.parametrize("rot,interleaved", [(128, False), (48, True), (0, False)])
def test_norm_rope_backward_against_differences(rot, interleaved):
    # directional derivatives of the plain 64-bit forward, central differences
    import gated_delta_rule_17_gb300 as gdn

    c = _norm_case(16, 9, 3, 2, 128, rot, F32, interleaved)
    at = c["pos"].long()
    cos, sin = (None, None) if not rot else (c["cos"][at], c["sin"][at])
    dq, dk = torch.empty(9, 3 * 128, device="cuda"), torch.empty(9, 2 * 128, device="cuda")
    dqw, dkw = torch.empty(128, device="cuda"), torch.empty(128, device="cuda")
    gdn.head_norm_rope_backward(c["q"].cuda().flatten(1), c["k"].cuda().flatten(1), c["pos"].cuda(), _cuda(c["cos"]), _cuda(c["sin"]),
                                c["gq"].cuda().flatten(1), c["gk"].cuda().flatten(1), dq, dk, dqw, dkw, nq=3, nkv=2,
                                q_weight=c["qw"].cuda(), k_weight=c["kw"].cuda(), interleaved=interleaved)
    gdn.check()

    def loss(q, k, qw, kw):
        return float((ref.norm_rope(q, qw, cos, sin, 1e-6, interleaved) * c["gq"].double()).sum()
                     + (ref.norm_rope(k, kw, cos, sin, 1e-6, interleaved) * c["gk"].double()).sum())

    x = [c["q"].double(), c["k"].double(), c["qw"].double(), c["kw"].double()]
    grads = [dq.cpu().double().view(9, 3, 128), dk.cpu().double().view(9, 2, 128), dqw.cpu().double(), dkw.cpu().double()]
    g = gen(17)
    h = 1e-4
    for i in range(4):
        way = torch.randn(x[i].shape, generator=g, dtype=torch.float64)
        there = [a + h * way if j == i else a for j, a in enumerate(x)]
        back = [a - h * way if j == i else a for j, a in enumerate(x)]
        slope = (loss(*there) - loss(*back)) / (2 * h)
        # h^2 third derivatives, and fp32 gradients summed over the direction
        assert abs(slope - float((grads[i] * way).sum())) <= 1e-5 * float((grads[i] * way).abs().sum())


def test_norm_rope_backward_in_place():
    import gated_delta_rule_17_gb300 as gdn

    c = _norm_case(18, 40, 4, 2, 64, 32, BF, False)
    q, k, gq, gk = (c[n].cuda().flatten(1) for n in ("q", "k", "gq", "gk"))
    dq, dk = torch.empty_like(q), torch.empty_like(k)
    kw = dict(nq=4, nkv=2, head_dim=64, q_weight=c["qw"].cuda(), k_weight=c["kw"].cuda())
    a = (q, k, c["pos"].cuda(), c["cos"].cuda(), c["sin"].cuda())
    gdn.head_norm_rope_backward(*a, gq, gk, dq, dk, **kw)
    gdn.head_norm_rope_backward(*a, gq, gk, gq, gk, **kw)
    gdn.check()
    assert torch.equal(dq, gq) and torch.equal(dk, gk)
    w = torch.full((64,), 3.0, device="cuda")
    gdn.head_norm_rope_backward(q[:0], k[:0], a[2][:0], *a[3:], gq[:0], gk[:0], dq[:0], dk[:0], w, **kw)
    assert (w == 0).all()  # the sum over no rows


# ---- the paged cache -------------------------------------------------------------------


class Cache:
    """Sequences of ctx[b] + new[b] tokens in a paged cache whose pages are in random order."""

    def __init__(self, seed, ctx, new, nkv, d, page, dtype, layout="tokens", spare=3, fill=None, far=0):
        g = gen(seed)
        self.g, self.ctx, self.new, self.nkv, self.d, self.page, self.dtype = g, ctx, new, nkv, d, page, dtype
        need = [-(-(a + n) // page) for a, n in zip(ctx, new)]
        pages = sum(need) + spare + far
        order = far + torch.randperm(sum(need) + spare, generator=g)
        most = max(max(need), 1)
        self.table = torch.full((len(ctx), most), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n].int()
            at += n
        if layout == "tokens":  # [pages, page, heads, d]
            kc = torch.empty(pages, page, nkv, d, dtype=dtype, device="cuda")
            vc = torch.empty(pages, page, nkv, d, dtype=dtype, device="cuda")
        elif layout == "heads":  # [pages, heads, page, d]
            kc = torch.empty(pages, nkv, page, d, dtype=dtype, device="cuda").transpose(1, 2)
            vc = torch.empty(pages, nkv, page, d, dtype=dtype, device="cuda").transpose(1, 2)
        else:  # keys and values side by side, with a gap after each page
            both = torch.empty(pages, page + 1, 2, nkv, d, dtype=dtype, device="cuda")
            kc, vc = both[:, :page, 0], both[:, :page, 1]
        self.kc, self.vc = kc, vc
        if fill is not None and far == 0:
            kc.fill_(fill)
            vc.fill_(fill)
        self.cu = torch.tensor([0] + [sum(new[:i + 1]) for i in range(len(new))], dtype=torch.int32)
        self.rows = sum(new)

    def place(self, b, t):
        return int(self.table[b, t // self.page]), t % self.page

    def fill_tokens(self):
        """Random keys and values for every token; returns them as [tokens, nkv, d] per sequence."""
        ks, vs = [], []
        for b, (a, n) in enumerate(zip(self.ctx, self.new)):
            k, v = randn(self.g, a + n, self.nkv, self.d, dtype=self.dtype), randn(self.g, a + n, self.nkv, self.d, dtype=self.dtype)
            t = torch.arange(a + n)
            pages = self.table[b].long()[t // self.page].cuda()
            self.kc[pages, (t % self.page).cuda()] = k.cuda()
            self.vc[pages, (t % self.page).cuda()] = v.cuda()
            ks.append(k)
            vs.append(v)
        return ks, vs

    def plan(self):
        return self.kc, self.vc, self.table.cuda(), torch.tensor(self.ctx, dtype=torch.int32, device="cuda")


APPEND_CASES = [
    dict(ctx=[0], new=[1], nkv=1, d=128, page=16, dtype=BF, rot=128),
    dict(ctx=[5, 0, 130], new=[7, 1, 33], nkv=3, d=128, page=17, dtype=BF, rot=128, layout="heads"),
    dict(ctx=[63, 64, 65], new=[2, 0, 130], nkv=8, d=64, page=64, dtype=HF, rot=32, inter=True, layout="side"),
    dict(ctx=[3, 900], new=[700, 1], nkv=5, d=128, page=1, dtype=HF, rot=48, norm=True),
    dict(ctx=[10] * 200, new=[i % 4 for i in range(200)], nkv=2, d=128, page=16, dtype=BF, rot=128, norm=True, weight=True),
    dict(ctx=[9, 8], new=[1, 1], nkv=9, d=64, page=256, dtype=BF, rot=0, norm=True, weight=True, no_cu=True),
]


@pytest.mark.parametrize("case", APPEND_CASES, ids=[str(i) for i in range(len(APPEND_CASES))])
@pytest.mark.parametrize("depths", [False, True])
def test_paged_append(case, depths):
    import gated_delta_rule_17_gb300 as gdn

    case = dict(case)
    rot, inter, norm, weight, no_cu = (case.pop(n, f) for n, f in (("rot", 0), ("inter", False), ("norm", False), ("weight", False), ("no_cu", False)))
    c = Cache(21, fill=-3.0, **case)
    g = c.g
    k, v = randn(g, c.rows, c.nkv, c.d, dtype=c.dtype), randn(g, c.rows, c.nkv, c.d, dtype=c.dtype)
    w = 1 + 0.2 * torch.randn(c.d, generator=g) if weight else None
    span = max(a + n for a, n in zip(c.ctx, c.new)) + 1
    cos, sin = ref.rope_tables(span, rot) if rot else (None, None)
    tokens = torch.cat([torch.arange(a, a + n) for a, n in zip(c.ctx, c.new)])
    pos = torch.randint(0, span, (c.rows,), generator=g, dtype=torch.int32) if depths else None
    kc, vc, table, lens = c.plan()
    gdn.paged_append(padded(k, 8), padded(v, 16), kc, vc, table, lens, nkv=c.nkv, head_dim=c.d,
                     cu_rows=None if no_cu else c.cu.cuda(), positions=_cuda(pos), cos=_cuda(cos), sin=_cuda(sin), norm=norm,
                     k_weight=_cuda(w), interleaved=inter)
    assert gdn.last_launch_count() == 1
    gdn.check()
    at = tokens if pos is None else pos.long()
    args = (w, None if cos is None else cos[at], None if sin is None else sin[at], 1e-6, inter, norm)
    want = ref.norm_rope(k.double(), *args)
    z = ref.norm_rope(k.double(), w, None, None, 1e-6, inter, norm)
    bound = ref.ROUNDING[c.dtype] * want.abs() + 32 * ref.FP32 * (ref.rotate_sizes(z, rot, inter) if rot else z.abs()) + 2.0 ** -25
    seq = torch.repeat_interleave(torch.arange(len(c.new)), torch.tensor(c.new))
    pages, place = c.table.long()[seq, tokens // c.page], tokens % c.page
    kh, vh = kc.cpu(), vc.cpu()
    assert ((kh[pages, place].double() - want).abs() <= bound).all()
    assert torch.equal(vh[pages, place], v)
    kh[pages, place] = -3.0  # nothing else is written
    vh[pages, place] = -3.0
    assert (kh == -3.0).all() and (vh == -3.0).all()


def test_paged_append_reports_bad_input():
    import gated_delta_rule_17_gb300 as gdn

    def call(c, cu=None, table=None, ctx=None, pos=None):
        kc, vc, tab, lens = c.plan()
        k = torch.ones(c.rows, c.nkv * c.d, dtype=c.dtype, device="cuda")
        cos, sin = ref.rope_tables(64, 128)
        gdn.paged_append(k, k, kc, vc, tab if table is None else table.cuda(), lens if ctx is None else ctx.cuda(), nkv=c.nkv,
                         cu_rows=(c.cu if cu is None else cu).cuda(), positions=_cuda(pos), cos=cos.cuda(), sin=sin.cuda())
        with pytest.raises(gdn.GdnError) as e:
            gdn.check()
        assert e.value.code == gdn.GDN_ERR_DEVICE_STATUS
        return str(e.value), (c.kc == -3.0).all(-1).all(-1).cpu(), (c.vc == -3.0).all(-1).all(-1).cpu()

    def cache():
        return Cache(22, [4, 20], [3, 2], 2, 128, 8, BF, fill=-3.0)

    c = cache()
    table = c.table.clone()
    table[0, 0] = 10 ** 6  # tokens 4 .. 6 of sequence 0
    msg, k_same, v_same = call(c, table=table)
    assert "page" in msg and int((~k_same).sum()) == 2 and int((~v_same).sum()) == 2
    c = cache()
    msg, k_same, _ = call(c, ctx=torch.tensor([4, 500], dtype=torch.int32))  # past the table
    assert "page" in msg and int((~k_same).sum()) == 3
    c = cache()
    msg, k_same, _ = call(c, ctx=torch.tensor([-4, 20], dtype=torch.int32))
    assert "malformed" in msg and int((~k_same).sum()) == 2
    c = cache()
    msg, k_same, _ = call(c, cu=torch.tensor([0, 3, 4], dtype=torch.int32))  # row 4 has no owner
    assert "malformed" in msg and int((~k_same).sum()) == 4
    c = cache()
    msg, k_same, v_same = call(c, pos=torch.tensor([0, 64, 1, 2, -1], dtype=torch.int32))
    assert "position" in msg and int((~k_same).sum()) == 3 and torch.equal(k_same, v_same)


# ---- attention -------------------------------------------------------------------------


def _tree(g, n):
    """A random draft tree: each row sees itself and its ancestors."""
    m = torch.zeros(n, n, dtype=torch.bool)
    for i in range(n):
        parent = int(torch.randint(-1, i, (1,), generator=g)) if i else -1
        if parent >= 0:
            m[i] = m[parent]
        m[i, i] = True
    return m


def _words(masks, rows):
    bits = max(max(m.shape[1] for m in masks), 1)
    full = torch.zeros(rows, bits, dtype=torch.bool)
    at = 0
    for m in masks:
        full[at:at + m.shape[0], :m.shape[1]] = m
        at += m.shape[0]
    return ref.pack_mask(full)


def _check_attention(c, q, out, ks, vs, masks, scale, rows_of=None):
    at = 0
    for b, (a, n) in enumerate(zip(c.ctx, c.new)):
        if rows_of is None or b in rows_of:
            want, spread, slack = ref.attention(q[at:at + n].double(), ks[b].double(), vs[b].double(), a,
                                                None if masks is None else masks[b], scale)
            bound = ref.attention_bound(want, spread, slack, c.dtype, a + n, float(vs[b].abs().max()) if a + n else 0.0)
            err = (out[at:at + n].double().view_as(want) - want).abs()
            assert (err <= bound).all(), (b, float((err / bound).max()))
        at += n


ATTEND_CASES = [
    # one token and no context; one token over one, over a page's end, over a tile's end
    dict(ctx=[0], new=[1], nq=1, nkv=1, d=128, page=16, dtype=BF),
    dict(ctx=[1, 15, 16, 63, 64, 127, 128, 257], new=[1] * 8, nq=8, nkv=2, d=128, page=16, dtype=BF),
    dict(ctx=[300, 0, 77], new=[1, 1, 1], nq=15, nkv=3, d=64, page=17, dtype=HF, layout="heads"),
    # trees, ragged, sequences without rows; groups of 1, 3, 8 and 16 heads
    dict(ctx=[40, 0, 500], new=[3, 5, 16], nq=4, nkv=4, d=128, page=64, dtype=BF, tree=True),
    dict(ctx=[40, 10, 0, 333], new=[7, 0, 64, 1], nq=6, nkv=2, d=128, page=16, dtype=HF, tree=True, layout="side"),
    dict(ctx=[130, 999], new=[33, 20], nq=16, nkv=2, d=64, page=16, dtype=BF, tree=True),
    dict(ctx=[200], new=[70], nq=16, nkv=1, d=128, page=1, dtype=BF, tree=True),
    dict(ctx=[700, 128], new=[130, 66], nq=8, nkv=2, d=128, page=256, dtype=BF, tree=True),
    # up to itself: a chunk of a prompt
    dict(ctx=[0, 100], new=[150, 40], nq=4, nkv=2, d=128, page=64, dtype=HF),
    dict(ctx=[31], new=[129], nq=5, nkv=1, d=64, page=17, dtype=BF),
    # many short sequences, and one long one that fills the card alone
    dict(ctx=[(7 * i) % 90 for i in range(300)], new=[1] * 300, nq=4, nkv=2, d=128, page=16, dtype=BF),
    dict(ctx=[20001], new=[1], nq=4, nkv=1, d=128, page=64, dtype=BF),
    dict(ctx=[9000], new=[5], nq=8, nkv=2, d=64, page=64, dtype=HF, tree=True),
    dict(ctx=[6000, 3], new=[40, 40], nq=8, nkv=2, d=128, page=64, dtype=BF, tree=True),
]


@pytest.mark.parametrize("case", ATTEND_CASES, ids=[str(i) for i in range(len(ATTEND_CASES))])
@pytest.mark.parametrize("hint", ["exact", "none"])
def test_tree_attention(case, hint):
    import gated_delta_rule_17_gb300 as gdn

    case = dict(case)
    nq, tree = case.pop("nq"), case.pop("tree", False)
    c = Cache(31, fill=float("nan"), **case)  # what lies past a sequence's tokens is NaN
    ks, vs = c.fill_tokens()
    q = 1.5 * randn(c.g, c.rows, nq, c.d, dtype=F32)
    q = q.to(c.dtype)
    masks = [_tree(c.g, n) for n in c.new] if tree else None
    scale = c.d ** -0.5
    qd, out = padded(q, 8), padded(torch.zeros_like(q), 24)
    kw = dict(nq=nq, nkv=c.nkv, head_dim=c.d, cu_rows=c.cu.cuda(), mask=_words(masks, c.rows).cuda() if tree else None)
    ws = torch.empty(gdn.tree_attention_workspace_bytes(nq, c.nkv, c.d), dtype=torch.uint8, device="cuda").fill_(255)
    gdn.tree_attention(qd, *c.plan(), out, workspace=ws if hint == "exact" else None,
                       max_rows=max(c.new) if hint == "exact" else None, **kw)
    assert 1 <= gdn.last_launch_count() <= 2
    gdn.check()
    assert torch.isnan(out._base[:, nq * c.d:]).all()
    got = out.cpu()
    _check_attention(c, q, got, ks, vs, masks, scale, rows_of=None if len(c.ctx) < 50 else range(0, 300, 7))
    # the same bits again
    again = torch.empty_like(got, device="cuda")
    gdn.tree_attention(qd, *c.plan(), again, workspace=ws, max_rows=max(c.new) if hint == "exact" else None, **kw)
    assert torch.equal(again.cpu(), got)


# Long sequences among many short ones: a CTA's share may end in front of a sequence's first tile, hold many
# whole sequences, or a part of one; a row is joined from few parts or from many, by one warp or by several.
UNEVEN_CASES = [
    dict(ctx=[3000] + [(13 * i) % 200 for i in range(120)] + [2500], new=[1] * 122, nq=8, nkv=2, d=128, page=64, dtype=BF),
    dict(ctx=[(29 * i) % 500 for i in range(40)] + [5000], new=[2] * 41, nq=8, nkv=8, d=64, page=16, dtype=HF),
    dict(ctx=[2100] + [(17 * i) % 300 for i in range(30)], new=[20] * 31, nq=8, nkv=1, d=128, page=64, dtype=BF),
    dict(ctx=[2600, 10, 2300], new=[40, 40, 33], nq=16, nkv=1, d=128, page=32, dtype=HF),
    dict(ctx=[5, 12000], new=[1, 9], nq=9, nkv=1, d=64, page=64, dtype=BF),
]


@pytest.mark.parametrize("case", UNEVEN_CASES, ids=[str(i) for i in range(len(UNEVEN_CASES))])
def test_uneven_sequences(case):
    import gated_delta_rule_17_gb300 as gdn

    case = dict(case)
    nq = case.pop("nq")
    c = Cache(47, fill=float("nan"), **case)
    ks, vs = c.fill_tokens()
    q = (1.5 * randn(c.g, c.rows, nq, c.d, dtype=F32)).to(c.dtype)
    masks = [_tree(c.g, n) for n in c.new]
    out = torch.full_like(q, float("nan"), device="cuda")
    gdn.tree_attention(q.cuda(), *c.plan(), out, nq=nq, nkv=c.nkv, head_dim=c.d, cu_rows=c.cu.cuda(), max_rows=max(c.new),
                       mask=_words(masks, c.rows).cuda())
    assert gdn.last_launch_count() == 2  # cut and joined
    gdn.check()
    _check_attention(c, q, out.cpu(), ks, vs, masks, c.d ** -0.5)


def test_tree_attention_without_cu_rows():
    import gated_delta_rule_17_gb300 as gdn

    c = Cache(32, [5, 70, 0], [1, 1, 1], 2, 128, 16, BF)
    ks, vs = c.fill_tokens()
    q = randn(c.g, 3, 6, 128)
    out = torch.empty(3, 6, 128, dtype=BF, device="cuda")
    gdn.tree_attention(q.cuda(), *c.plan(), out, nq=6, nkv=2, scale=0.3)
    gdn.check()
    _check_attention(c, q, out.cpu(), ks, vs, None, 0.3)


@pytest.mark.parametrize("n", [3, 40, 130])
def test_rows_that_see_nothing_give_zeros(n):
    import gated_delta_rule_17_gb300 as gdn

    c = Cache(33, [0, 9], [n, n], 2, 128, 16, BF)
    ks, vs = c.fill_tokens()
    q = randn(c.g, c.rows, 8, 128)
    masks = [_tree(c.g, n), _tree(c.g, n)]
    masks[0][1] = False
    masks[0][n - 1] = False
    masks[1][0] = False
    masks[1][2, :] = True  # a row may see later rows too
    out = torch.full((c.rows, 8 * 128), float("nan"), dtype=BF, device="cuda")
    gdn.tree_attention(q.cuda(), *c.plan(), out, nq=8, nkv=2, cu_rows=c.cu.cuda(), mask=_words(masks, c.rows).cuda(), max_rows=n)
    gdn.check()
    got = out.cpu()
    assert (got[1] == 0).all() and (got[n - 1] == 0).all()
    _check_attention(c, q, got, ks, vs, masks, 128 ** -0.5)


def test_mask_words_that_do_not_reach():
    # 70 rows with one word: rows 64 .. 69 are seen by none
    import gated_delta_rule_17_gb300 as gdn

    c = Cache(34, [20], [70], 1, 64, 16, HF)
    ks, vs = c.fill_tokens()
    q = randn(c.g, 70, 2, 64, dtype=HF)
    mask = _tree(c.g, 70)
    mask[:, 64:] = False
    out = torch.empty(70, 128, dtype=HF, device="cuda")
    gdn.tree_attention(q.cuda(), *c.plan(), out, nq=2, nkv=1, head_dim=64, cu_rows=c.cu.cuda(), mask=_words([mask[:, :64]], 70).cuda())
    gdn.check()
    _check_attention(c, q, out.cpu(), ks, vs, [mask], 0.125)


@pytest.mark.parametrize("n", [1, 24])
def test_scores_far_apart(n):
    # scores of +-1000: the running maximum jumps, nearly all weights are 0 or 1
    import gated_delta_rule_17_gb300 as gdn

    c = Cache(35, [700, 90], [n, n], 2, 128, 16, BF)
    ks, vs = c.fill_tokens()
    q = (60 * torch.randn(c.rows, 8, 128, generator=c.g)).to(BF)
    out = torch.empty(c.rows, 8 * 128, dtype=BF, device="cuda")
    gdn.tree_attention(q.cuda(), *c.plan(), out, nq=8, nkv=2, cu_rows=c.cu.cuda(), max_rows=n)
    gdn.check()
    assert torch.isfinite(out).all()
    _check_attention(c, q, out.cpu(), ks, vs, None, 128 ** -0.5)


@pytest.mark.parametrize("scale", [-0.1, 0.0, 1e-30, 5.0])
@pytest.mark.parametrize("n", [2, 30])
def test_any_scale(n, scale):
    import gated_delta_rule_17_gb300 as gdn

    c = Cache(40, [300, 50], [n, n], 2, 128, 16, BF)
    ks, vs = c.fill_tokens()
    q = randn(c.g, c.rows, 8, 128)
    out = torch.empty(c.rows, 8 * 128, dtype=BF, device="cuda")
    gdn.tree_attention(q.cuda(), *c.plan(), out, nq=8, nkv=2, cu_rows=c.cu.cuda(), max_rows=n, scale=scale)
    gdn.check()
    _check_attention(c, q, out.cpu(), ks, vs, None, scale)


def test_output_rows_on_16_byte_boundaries():
    # rows that whole 32-byte sectors do not fit; on tcgen05 and not
    import gated_delta_rule_17_gb300 as gdn

    for n in (3, 40):
        c = Cache(41, [70, 0], [n, n], 2, 64, 16, HF)
        ks, vs = c.fill_tokens()
        q = randn(c.g, c.rows, 8, 64, dtype=HF)
        wide = torch.full((c.rows, 8 * 64 + 24), 9.0, dtype=HF, device="cuda")
        out = wide[:, 8:8 + 8 * 64]
        gdn.tree_attention(q.cuda(), *c.plan(), out, nq=8, nkv=2, head_dim=64, cu_rows=c.cu.cuda(), max_rows=n)
        gdn.check()
        _check_attention(c, q, out.cpu(), ks, vs, None, 0.125)
        assert (wide[:, :8] == 9).all() and (wide[:, 8 + 8 * 64:] == 9).all()


@pytest.mark.parametrize("n", [1, 20])
def test_cache_past_four_gigabytes(n):
    # pages whose first element is past 2^31: 64-bit offsets, in the append and the attention
    import gated_delta_rule_17_gb300 as gdn

    page, nkv, d = 64, 8, 128
    far = (1 << 31) // (page * nkv * d) + 1
    c = Cache(36, [150, 70], [n, n], nkv, d, page, BF, far=far)
    assert int(c.table[0, 0]) * c.kc.stride(0) > 1 << 31
    ks, vs = c.fill_tokens()
    at = 0
    k, v = torch.cat([x[a:] for x, a in zip(ks, c.ctx)]), torch.cat([x[a:] for x, a in zip(vs, c.ctx)])
    kc, vc, table, lens = c.plan()
    for b, a in enumerate(c.ctx):  # the new tokens come through the append
        for t in range(a, a + n):
            p, o = c.place(b, t)
            kc[p, o] = 0
            vc[p, o] = 0
            at += 1
    gdn.paged_append(k.cuda().flatten(1), v.cuda().flatten(1), kc, vc, table, lens, nkv=nkv, cu_rows=c.cu.cuda())
    q = randn(c.g, c.rows, 16, d)
    out = torch.empty(c.rows, 16 * d, dtype=BF, device="cuda")
    gdn.tree_attention(q.cuda(), kc, vc, table, lens, out, nq=16, nkv=nkv, cu_rows=c.cu.cuda(), max_rows=n)
    gdn.check()
    _check_attention(c, q, out.cpu(), ks, vs, None, d ** -0.5)


def test_on_another_stream():
    # everything on one side stream, without a synchronisation in between
    import gated_delta_rule_17_gb300 as gdn

    c = Cache(37, [100, 40], [6, 3], 2, 128, 16, BF, fill=0.0)
    ks, vs = c.fill_tokens()
    cu, plan = c.cu.cuda(), c.plan()
    q = randn(c.g, c.rows, 8, 128)
    k, v = torch.cat([x[a:] for x, a in zip(ks, c.ctx)]), torch.cat([x[a:] for x, a in zip(vs, c.ctx)])
    k, v, qd = k.cuda().flatten(1), v.cuda().flatten(1), q.cuda()
    out = torch.empty(c.rows, 8 * 128, dtype=BF, device="cuda")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    gdn.paged_append(k, v, *plan, nkv=2, cu_rows=cu, stream=s)
    gdn.tree_attention(qd, *plan, out, nq=8, nkv=2, cu_rows=cu, stream=s)
    gdn.check(s)
    _check_attention(c, q, out.cpu(), ks, vs, None, 128 ** -0.5)


def test_in_a_graph():
    # captured once with a kept workspace, replayed over a context that has grown meanwhile
    import gated_delta_rule_17_gb300 as gdn

    c = Cache(38, [200, 90], [30, 30], 2, 128, 16, BF)
    ks, vs = c.fill_tokens()
    kc, vc, table, _ = c.plan()
    lens = torch.tensor([10, 20], dtype=torch.int32, device="cuda")
    q = randn(c.g, 2, 8, 128).cuda()
    out = torch.empty(2, 8 * 128, dtype=BF, device="cuda")
    ws = torch.empty(gdn.tree_attention_workspace_bytes(8, 2), dtype=torch.uint8, device="cuda")
    call = lambda: gdn.tree_attention(q, kc, vc, table, lens, out, nq=8, nkv=2, workspace=ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for a in ([10, 20], [229, 0], [64, 119]):
        lens.copy_(torch.tensor(a, dtype=torch.int32))
        out.zero_()
        graph.replay()
        gdn.check()
        d = Cache.__new__(Cache)
        d.ctx, d.new, d.dtype = a, [1, 1], BF
        _check_attention(d, q.cpu(), out.cpu(), [k[:x + 1] for k, x in zip(ks, a)], [v[:x + 1] for v, x in zip(vs, a)], None, 128 ** -0.5)


def test_tree_attention_reports_bad_input():
    import gated_delta_rule_17_gb300 as gdn

    def call(c, q, cu=None, table=None, ctx=None):
        kc, vc, tab, lens = c.plan()
        out = torch.full((c.rows, 4 * 128), 7.0, dtype=BF, device="cuda")
        gdn.tree_attention(q.cuda(), kc, vc, tab if table is None else table.cuda(), lens if ctx is None else ctx.cuda(), out, nq=4, nkv=2,
                           cu_rows=(c.cu if cu is None else cu).cuda())
        with pytest.raises(gdn.GdnError) as e:
            gdn.check()
        assert e.value.code == gdn.GDN_ERR_DEVICE_STATUS
        return str(e.value), out.cpu()

    c = Cache(39, [40, 20], [3, 2], 2, 128, 8, BF)
    ks, vs = c.fill_tokens()
    q = randn(c.g, 5, 4, 128)
    table = c.table.clone()
    table[0, 1] = 10 ** 6  # tokens 8 .. 15 are not there: zeros to the attention
    msg, out = call(c, q, table=table)
    assert "page" in msg
    there = ((torch.arange(43) < 8) | (torch.arange(43) >= 16))[:, None, None]
    _check_attention(c, q, out, [ks[0] * there, ks[1]], [vs[0] * there, vs[1]], None, 128 ** -0.5)
    msg, out = call(c, q, ctx=torch.tensor([-1, 20], dtype=torch.int32))
    assert "malformed" in msg and (out[:3] == 7.0).all()
    msg, out = call(c, q, cu=torch.tensor([0, 9, 5], dtype=torch.int32))
    assert "malformed" in msg and (out == 7.0).all()
    msg, out = call(c, q, ctx=torch.tensor([40, 10 ** 6], dtype=torch.int32))
    assert "page" in msg
    # and the next call is sound
    kc, vc, tab, lens = c.plan()
    out = torch.empty(5, 4 * 128, dtype=BF, device="cuda")
    gdn.tree_attention(q.cuda(), kc, vc, tab, lens, out, nq=4, nkv=2, cu_rows=c.cu.cuda())
    gdn.check()
    _check_attention(c, q, out.cpu(), ks, vs, None, 128 ** -0.5)
