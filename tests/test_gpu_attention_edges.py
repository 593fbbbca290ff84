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
