"""GPU tests of the softmax-attention operators at sizes and values where their arithmetic or their schedule could go
wrong, against plain 64-bit forms, with bounds that follow from the kernels' roundings."""
import pytest

torch = pytest.importorskip("torch")

from tests import attention_reference as ref  # noqa: E402
from tests.test_gpu_attention import BF, F32, HF, Cache, _built, _check_attention, _cuda, gen, padded, randn  # noqa: E402, F401

pytestmark = pytest.mark.gpu


# ---- the backward of norm and rotation -----------------------------------------------------


def _backward(x, dy, w, cos, sin, pos, eps, interleaved=False):
    """dq and the weight's gradient of q alone, x and dy [rows, heads, d] on the host."""
    import gated_delta_rule_17_gb300 as gdn

    rows, heads, d = x.shape
    dx, dw = torch.empty(rows, heads * d, dtype=x.dtype, device="cuda"), torch.empty(d, device="cuda")
    gdn.head_norm_rope_backward(x.cuda().flatten(1), None, _cuda(pos), _cuda(cos), _cuda(sin), dy.cuda().flatten(1), None, dx, None, dw,
                                nq=heads, nkv=0, head_dim=d, q_weight=_cuda(w), eps=eps, interleaved=interleaved)
    gdn.check()
    return dx.cpu().double().view(rows, heads, d), dw.cpu().double()


# rows of these sizes: the sum of their squares is inside fp32, the cube of their root mean square is not
@pytest.mark.parametrize("size,eps", [(1e12, 1e-6), (1e15, 1e-6), (1e17, 1e-6), (1e-13, 0.0), (1e-15, 0.0)])
@pytest.mark.parametrize("dtype,rot", [(F32, 0), (F32, 128), (BF, 128)])
def test_norm_rope_backward_of_rows_of_any_size(size, eps, dtype, rot):
    g = gen(61)
    x, dy = (size * randn(g, 6, 3, 128, dtype=F32)).to(dtype), randn(g, 6, 3, 128, dtype=dtype)
    w = 1 + 0.2 * torch.randn(128, generator=g)
    cos, sin = ref.rope_tables(9, rot) if rot else (None, None)
    pos = torch.randint(0, 9, (6,), generator=g, dtype=torch.int32)
    got, gotw = _backward(x, dy, w, cos, sin, pos, eps)
    at = pos.long()
    want, wsum, wsize, room = ref.norm_rope_backward(x.double(), dy.double(), w, None if cos is None else cos[at],
                                                     None if sin is None else sin[at], eps, False)
    # fp32: two row sums (<= 16 additions in a chain), rsqrt, about ten products and sums
    bound = ref.ROUNDING[dtype] * want.abs() + 64 * ref.FP32 * room
    assert ((got - want).abs() <= bound).all(), float(((got - want).abs() / bound).max())
    # 18 terms: each a rotated value, which is a difference of two, times x r; and their sum
    both = dy.double().abs() if cos is None else ref.rotate_sizes(dy.double(), rot, False)
    wroom = (both * x.double().abs() / torch.sqrt((x.double() ** 2).mean(-1, keepdim=True) + eps)).sum((0, 1))
    assert ((gotw - wsum).abs() <= (18 + 32) * ref.FP32 * wroom).all()


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("held", [50, 0])
def test_norm_rope_backward_of_positions_outside_the_table(dtype, held):
    # reported and left out, of the weights' gradients too; a table without rows is not read
    import ctypes

    import gated_delta_rule_17_gb300 as gdn

    g = gen(62)
    x, dy = randn(g, 12, 5, 128, dtype=dtype), randn(g, 12, 5, 128, dtype=dtype)
    cos, sin = ref.rope_tables(50, 128)
    pos = torch.randint(0, 50, (12,), generator=g, dtype=torch.int32)
    pos[3], pos[7] = 50, -1
    good = [i for i in range(12) if 0 <= pos[i] < held]
    dev = dict(x=x.cuda(), dy=dy.cuda(), cos=cos.cuda(), sin=sin.cuda(), pos=pos.cuda(), dx=torch.full_like(x, 7.0, device="cuda"),
               dw=torch.full((128,), float("nan"), device="cuda"))
    at = {n: t.data_ptr() for n, t in dev.items()}
    rope = gdn.Rope(at["cos"], at["sin"], 64, held, 128, 0)
    rc = gdn.load().gdn_head_norm_rope_backward(at["x"], None, at["pos"], ctypes.addressof(rope), None, None, 1e-6, at["dy"], None, at["dx"],
                                                None, at["dw"], None, 12, 5, 0, 128, 2 if dtype is F32 else 0, None, None, 0, 0)
    assert rc == gdn.GDN_OK
    with pytest.raises(gdn.GdnError) as e:
        gdn.check(0)
    assert e.value.code == gdn.GDN_ERR_DEVICE_STATUS and "position" in str(e.value)
    bad = [i for i in range(12) if i not in good]
    dx, dw = dev["dx"].cpu(), dev["dw"].cpu().double()
    assert (dx[bad] == 7.0).all()
    if not good:
        assert (dw == 0).all()
        return
    xs, ys, ps = x[good].double(), dy[good].double(), pos[good].long()
    want, wsum, _, room = ref.norm_rope_backward(xs, ys, None, cos[ps], sin[ps], 1e-6, False)
    assert ((dx[good].double() - want).abs() <= ref.ROUNDING[dtype] * want.abs() + 64 * ref.FP32 * room).all()
    wroom = (ref.rotate_sizes(ys, 128, False) * xs.abs() / torch.sqrt((xs ** 2).mean(-1, keepdim=True) + 1e-6)).sum((0, 1))
    assert ((dw - wsum).abs() <= (50 + 32) * ref.FP32 * wroom).all()


@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("rows,heads,d", [(1, 1, 128), (3, 7, 64), (40, 9, 128), (999, 3, 64), (1100, 12, 128), (2500, 32, 64)])
def test_no_row_is_lost_from_the_weight_gradients(rows, heads, d, dtype):
    # x of +-1 has r = 1 (up to rsqrt's two units in the last place), so that dw sums whole numbers, exactly
    g = gen(68)
    x = (torch.randint(0, 2, (rows, heads, d), generator=g) * 2 - 1).to(dtype)
    dy = torch.randint(1, 4, (rows, heads, d), generator=g).to(dtype) * x  # each term is 1, 2 or 3
    _, dw = _backward(x, dy, None, None, None, None, 0.0)
    want = (x.double() * dy.double()).sum((0, 1))
    # Where r is not quite 1: its two units, and the roundings of sums that are no whole numbers then. At the largest case
    # here a lane adds 8 head rows, a warp's lanes 2 more, 4 warps, 29 partials a warp of the last sum, 5 steps over these.
    assert ((dw - want).abs() <= (4 + 60) * ref.FP32 * want).all()
    assert float((4 + 60) * ref.FP32 * want.max()) < 1  # and no term is as small


# ---- attention -----------------------------------------------------------------------------


@pytest.mark.parametrize("peak", ["first", "last"])
@pytest.mark.parametrize("nq,n", [(1, 1), (8, 5)])
def test_fp16_sums_of_many_small_weights(nq, n, peak):
    # One token outweighs each of 40000 others by 2^26, and has a value of zero: what the others add up to, 0.06% of the
    # weight, is the output. As fp16 numbers below 1 their weights of 2^-26 would be gone. As many sequences (of the same
    # pages) as there are CTAs, so that one CTA has a sequence's tokens and one maximum for many of them.
    import gated_delta_rule_17_gb300 as gdn

    tokens, d, page = 40000, 64, 64
    B = torch.cuda.get_device_properties(0).multi_processor_count * (2 if nq * n <= 16 else 1)
    g = gen(64)
    k, v = torch.zeros(tokens, 1, d, dtype=HF), (256 + 128 * torch.rand(tokens, 1, d, generator=g)).to(HF)
    at = 0 if peak == "first" else tokens - n
    k[at, 0, 0] = 26 * 0.6931471805599453 * 8 / 4  # times q's 4 and 1 / sqrt(d): 26 in units of log 2
    v[at] = 0
    kc, vc = k.cuda().view(-1, page, 1, d), v.cuda().view(-1, page, 1, d)
    table = torch.arange(tokens // page, dtype=torch.int32, device="cuda").repeat(B, 1)
    lens = torch.full((B,), tokens - n, dtype=torch.int32, device="cuda")
    cu = torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda")
    q = torch.zeros(n, nq, d, dtype=HF)
    q[:, :, 0] = 4
    out = torch.empty(B * n, nq * d, dtype=HF, device="cuda")
    gdn.tree_attention(q.cuda().repeat(B, 1, 1), kc, vc, table, lens, out, nq=nq, nkv=1, head_dim=d, cu_rows=cu, max_rows=n)
    gdn.check()
    want, spread, slack = ref.attention(q.double(), k.double(), v.double(), tokens - n, None, 0.125)
    assert float(want.min()) > 0.15
    # u for the rounded output and u for the rounded weights, which are fractions of a row's largest, 2^6, or of more:
    # down to 2^-14 they have fp16's relative rounding, below they are off by up to 2^-25 of 2^6 each
    u = ref.ROUNDING[HF]
    bound = u * want.abs() + (u + slack) * spread * (1 + 2 * u) + (tokens + 1) * 2.0 ** -31 * float(v.abs().max()) + 2.0 ** -25
    err = (out.cpu().double().view(B, n, nq, d) - want).abs()
    assert (err <= bound).all(), float((err / bound).max())


def _attention_on_the_card(c, q, ks, vs, scale):
    """Causal attention of every row in 64 bits, and its error bound (as attention_reference.attention has it)."""
    wants, bounds, at = [], [], 0
    nq, group = q.shape[1], q.shape[1] // c.nkv
    for b, (a, n) in enumerate(zip(c.ctx, c.new)):
        want = torch.zeros(n, nq, c.d, dtype=torch.float64, device="cuda")
        bound = torch.zeros_like(want)
        unseen = torch.arange(a + n, device="cuda") > a + torch.arange(n, device="cuda")[:, None]
        for h in range(nq):
            k, v, qh = (x.double().cuda() for x in (ks[b][:, h // group], vs[b][:, h // group], q[at:at + n, h]))
            x = scale * (qh @ k.T)
            p = torch.softmax(x.masked_fill(unseen, float("-inf")), -1)
            want[:, h] = p @ v
            size = abs(scale) * (c.d + 4) * (qh.abs() @ k.abs().T).masked_fill(unseen, 0).amax(-1) + 4 * x.abs().masked_fill(unseen, 0).amax(-1)
            slack = 2 * ref.FP32 * (size[:, None] + a + n + 16)
            bound[:, h] = ref.attention_bound(want[:, h], p @ v.abs(), slack, c.dtype, a + n, float(v.abs().max()))
        wants.append(want)
        bounds.append(bound)
        at += n
    return torch.cat(wants), torch.cat(bounds)


# Chunks of a prompt with more row tiles of a kv head than there are groups of CTAs (8): a group then has several.
CHUNKS = [
    dict(ctx=[0], new=[700], nq=8, nkv=2, d=128, page=64, dtype=BF),  # 11 row tiles of 256, whole units
    dict(ctx=[3000, 10, 500], new=[560, 3, 1030], nq=4, nkv=1, d=128, page=16, dtype=BF),  # 9, 1 and 17, cut
    dict(ctx=[900], new=[2100], nq=2, nkv=1, d=64, page=24, dtype=HF),
]


@pytest.mark.parametrize("case", CHUNKS, ids=[str(i) for i in range(len(CHUNKS))])
@pytest.mark.parametrize("hint", ["exact", "too low"])
def test_many_row_tiles(case, hint):
    # max_rows below a sequence's rows: the kernel for few rows then has them in tiles of 16
    import gated_delta_rule_17_gb300 as gdn

    case = dict(case)
    nq = case.pop("nq")
    c = Cache(65, fill=float("nan"), **case)
    ks, vs = c.fill_tokens()
    q = (1.5 * randn(c.g, c.rows, nq, c.d, dtype=F32)).to(c.dtype)
    out = torch.full((c.rows, nq * c.d), float("nan"), dtype=c.dtype, device="cuda")
    gdn.tree_attention(q.cuda(), *c.plan(), out, nq=nq, nkv=c.nkv, head_dim=c.d, cu_rows=c.cu.cuda(),
                       max_rows=max(c.new) if hint == "exact" else 1)
    gdn.check()
    want, bound = _attention_on_the_card(c, q, ks, vs, c.d ** -0.5)
    err = (out.double().view_as(want) - want).abs()
    assert (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("page,d", [(8, 128), (24, 128), (40, 64), (48, 64)])
def test_pages_of_small_boxes_on_the_tensor_cores(page, d):
    # copies of 8 and 16 tokens inside the pages
    import gated_delta_rule_17_gb300 as gdn

    c = Cache(66, [500, 3, 129], [20, 33, 8], 2, d, page, BF, fill=float("nan"))
    ks, vs = c.fill_tokens()
    q = (1.5 * randn(c.g, c.rows, 8, d, dtype=F32)).to(BF)
    out = torch.empty(c.rows, 8 * d, dtype=BF, device="cuda")
    gdn.tree_attention(q.cuda(), *c.plan(), out, nq=8, nkv=2, head_dim=d, cu_rows=c.cu.cuda(), max_rows=33)
    gdn.check()
    _check_attention(c, q, out.cpu(), ks, vs, None, d ** -0.5)


@pytest.mark.parametrize("page", [8, 64])
@pytest.mark.parametrize("number", [-1, 10 ** 6])
def test_a_bad_page_on_the_tensor_cores(page, number):
    # its tokens have keys and values of zeros, and the status says so
    import gated_delta_rule_17_gb300 as gdn

    c = Cache(67, [300, 70], [20, 25], 2, 128, page, BF, fill=float("nan"))
    ks, vs = c.fill_tokens()
    q = randn(c.g, c.rows, 8, 128)
    kc, vc, table, lens = c.plan()
    table[0, 1] = number
    out = torch.empty(c.rows, 8 * 128, dtype=BF, device="cuda")
    gdn.tree_attention(q.cuda(), kc, vc, table, lens, out, nq=8, nkv=2, cu_rows=c.cu.cuda(), max_rows=25)
    with pytest.raises(gdn.GdnError) as e:
        gdn.check()
    assert e.value.code == gdn.GDN_ERR_DEVICE_STATUS and "page" in str(e.value)
    there = ((torch.arange(320) // page) != 1)[:, None, None]
    _check_attention(c, q, out.cpu(), [ks[0] * there, ks[1]], [vs[0] * there, vs[1]], None, 128 ** -0.5)
