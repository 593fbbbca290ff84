"""Calls that the operators around and beside the recurrence have to refuse, by name and before anything is launched. No GPU."""
import os
import re

import pytest

from tests.test_attention_refusals import OnCard, refused

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 256  # an aligned address that no check dereferences


@pytest.fixture(scope="module")
def gdn():
    from gated_delta_rule_17_gb300 import build

    build.build()
    import gated_delta_rule_17_gb300 as gdn

    gdn.load()
    return gdn


def test_every_declared_symbol_is_exported(gdn):
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "gdn_recurrent.h")).read(), flags=re.S)
    names = set(re.findall(r"^\s*(?:int|size_t)\s+(gdn_[a-z_0-9]+)\s*\(", src, flags=re.M))
    assert names == {"gdn_causal_conv", "gdn_causal_conv_backward", "gdn_causal_conv_backward_workspace_bytes", "gdn_ssm_scan",
                     "gdn_ssm_scan_workspace_bytes", "gdn_ssm_decode", "gdn_layer_norm", "gdn_layer_norm_backward",
                     "gdn_layer_norm_backward_workspace_bytes"}
    for n in names:
        assert hasattr(gdn.load(), n)


def test_internal_names_are_not_exported(gdn):
    import subprocess

    out = subprocess.run(["nm", "-D", "--defined-only", gdn.lib_path()], capture_output=True, text=True).stdout
    assert "gdn_causal_conv" in out and "gdn_host" not in out


def conv(gdn, x=P, w=P, b=P, state=P, out=2 * P, B=2, T=3, D=64, width=4, silu=1, dtype=0, table=0, xs=0, os_=0, cu=None):
    rc = gdn.load().gdn_causal_conv(x, w, b, state, out, B, T, D, width, silu, dtype, table, xs, os_, cu, None)
    return rc, gdn.load().gdn_last_error().decode()


def conv_back(gdn, x=P, w=P, b=P, h0=P, dout=2 * P, dST=P, dx=3 * P, dw=P, db=P, dh0=P, B=2, T=3, D=64, width=4, silu=1, dtype=0, xs=0, gs=0,
              ds=0, cu=None, ws=None, size=0):
    rc = gdn.load().gdn_causal_conv_backward(x, w, b, h0, dout, dST, dx, dw, db, dh0, B, T, D, width, silu, dtype, xs, gs, ds, cu, ws, size, None)
    return rc, gdn.load().gdn_last_error().decode()


BOTH = [
    ("ARG", "negative", dict(B=-1)), ("ARG", "negative", dict(T=-1)), ("UNSUPPORTED", "row range", dict(B=1 << 20, T=1 << 20)),
    ("UNSUPPORTED", "D = ", dict(D=0)), ("UNSUPPORTED", "D = ", dict(D=-8)), ("UNSUPPORTED", "D = ", dict(D=60)),
    ("UNSUPPORTED", "D = ", dict(D=(1 << 26) + 8)), ("UNSUPPORTED", "item range", dict(B=1 << 30, T=1, D=512)),
    ("UNSUPPORTED", "width", dict(width=1)), ("UNSUPPORTED", "width", dict(width=5)), ("UNSUPPORTED", "dtype", dict(dtype=3)),
    ("ARG", "silu", dict(silu=2)), ("ARG", "x row stride", dict(xs=56)), ("ARG", "x row stride", dict(xs=68)), ("ARG", "x row stride", dict(xs=-64)),
    ("ARG", "NULL", dict(w=None)), ("ARG", "NULL", dict(x=None)), ("ARG", "aligned", dict(x=P + 8)), ("ARG", "aligned", dict(w=P + 4)),
    ("ARG", "aligned", dict(b=P + 4)),
]


@pytest.mark.parametrize("code,words,kw", BOTH + [
    ("ARG", "out row stride", dict(os_=32)), ("ARG", "state_is_table", dict(table=2)), ("ARG", "table", dict(table=1, state=None)),
    ("ARG", "NULL", dict(out=None)), ("ARG", "must not be x", dict(out=P)), ("ARG", "aligned", dict(out=2 * P + 2)), ("ARG", "aligned", dict(state=P + 8)),
    ("ARG", "aligned", dict(state=P + 4, table=1)),
])
def test_conv_refusals(gdn, code, words, kw):
    rc, msg = conv(gdn, **kw)
    assert rc == getattr(gdn, "GDN_ERR_" + code) and words in msg, msg


@pytest.mark.parametrize("code,words,kw", BOTH + [
    ("ARG", "dout row stride", dict(gs=32)), ("ARG", "dx row stride", dict(ds=32)), ("ARG", "NULL", dict(dout=None)), ("ARG", "NULL", dict(dx=None)),
    ("ARG", "must not be x", dict(dx=P)), ("ARG", "must not be x", dict(dx=2 * P)), ("ARG", "aligned", dict(dout=P + 2)), ("ARG", "aligned", dict(h0=P + 8)),
    ("ARG", "aligned", dict(dST=P + 8)), ("ARG", "aligned", dict(dh0=P + 8)), ("ARG", "smaller", dict(ws=P, size=16)),
    ("ARG", "256-byte", dict(ws=P + 16, size=1 << 30)),
])
def test_conv_backward_refusals(gdn, code, words, kw):
    rc, msg = conv_back(gdn, **kw)
    assert rc == getattr(gdn, "GDN_ERR_" + code) and words in msg, msg


def ssm(gdn, q=P, k=P, v=P, dt=P, a=P, bias=P, skip=P, state=P, out=2 * P, B=2, T=3, nk=2, nv=4, dk=128, dv=64, o=None, cu=None, ws=None, size=0):
    lib = gdn.load()
    opt = gdn._SSM(*o) if o else None
    rc = lib.gdn_ssm_scan(q, k, v, dt, a, bias, skip, state, out, B, T, nk, nv, dk, dv, opt, cu, ws, size, None)
    return rc, lib.gdn_last_error().decode()


def step(gdn, q=P, k=P, v=P, dt=P, a=P, bias=P, skip=P, state=P, out=2 * P, B=2, nk=2, nv=4, dk=128, dv=64, o=None):
    lib = gdn.load()
    rc = lib.gdn_ssm_decode(q, k, v, dt, a, bias, skip, state, out, B, nk, nv, dk, dv, gdn._SSM(*o) if o else None, None)
    return rc, lib.gdn_last_error().decode()


OPT = [256, 256, 256, 4, 256, 0, 0, 1]


def opt(i, x):
    o = list(OPT)
    o[i] = x
    return o


@pytest.mark.parametrize("code,words,kw", [
    ("ARG", "negative", dict(B=-1)), ("ARG", "positive", dict(nk=0)), ("ARG", "positive", dict(nv=0)), ("UNSUPPORTED", "multiple of nk", dict(nv=3)),
    ("UNSUPPORTED", "row's range", dict(nk=1, nv=1 << 25)), ("UNSUPPORTED", "row's range", dict(nk=1 << 26, nv=1 << 26, dk=64)),
    ("UNSUPPORTED", "dk", dict(dk=96)), ("UNSUPPORTED", "dv", dict(dv=0)), ("UNSUPPORTED", "dv", dict(dv=256)),
    ("ARG", "q row stride", dict(o=opt(0, 128))), ("ARG", "k row stride", dict(o=opt(1, 260))), ("ARG", "v row stride", dict(o=opt(2, -8))),
    ("ARG", "dt row stride", dict(o=opt(3, 3))), ("ARG", "out row stride", dict(o=opt(4, 8))), ("ARG", "state_is_table", dict(o=opt(5, 2))),
    ("ARG", "dt_bf16", dict(o=opt(6, -1))), ("ARG", "softplus", dict(o=opt(7, 3))), ("ARG", "NULL", dict(q=None)), ("ARG", "NULL", dict(k=None)),
    ("ARG", "NULL", dict(v=None)), ("ARG", "NULL", dict(dt=None)), ("ARG", "NULL", dict(a=None)), ("ARG", "NULL", dict(state=None)),
    ("ARG", "NULL", dict(out=None)), ("ARG", "aligned", dict(v=P + 8)), ("ARG", "aligned", dict(state=P + 8)), ("ARG", "aligned", dict(dt=P + 2)),
    ("ARG", "aligned", dict(skip=P + 1)), ("ARG", "aligned", dict(dt=P + 1, o=opt(6, 1))),
])
def test_ssm_refusals(gdn, code, words, kw):
    for f in (ssm, step):
        rc, msg = f(gdn, **kw)
        assert rc == getattr(gdn, "GDN_ERR_" + code) and words in msg, msg


def test_scan_refuses_its_inputs_as_output(gdn):
    for name in ("q", "k", "v"):
        rc, msg = ssm(gdn, **{name: 2 * P})
        assert rc == gdn.GDN_ERR_ARG and "must not be" in msg
    assert ssm(gdn, B=1 << 20, T=1 << 20)[0] == gdn.GDN_ERR_UNSUPPORTED


def ln(gdn, x=P, z=None, w=P, b=P, eps=1e-5, out=2 * P, rows=3, groups=2, dim=64, dtype=0, rms=0, first=0, st=None):
    rc = gdn.load().gdn_layer_norm(x, z, w, b, eps, out, rows, groups, dim, dtype, rms, first, gdn._LAYER_NORM(*st) if st else None, None)
    return rc, gdn.load().gdn_last_error().decode()


def ln_back(gdn, x=P, z=None, w=P, b=P, eps=1e-5, dout=2 * P, dx=3 * P, dz=None, dw=P, db=P, rows=3, groups=2, dim=64, dtype=0, rms=0, first=0,
            st=None, ws=None, size=0):
    rc = gdn.load().gdn_layer_norm_backward(x, z, w, b, eps, dout, dx, dz, dw, db, rows, groups, dim, dtype, rms, first,
                                            gdn._LAYER_NORM(*st) if st else None, ws, size, None)
    return rc, gdn.load().gdn_last_error().decode()


NORMS = [
    ("ARG", "rows", dict(rows=-1)), ("ARG", "groups", dict(groups=0)), ("UNSUPPORTED", "dim", dict(dim=0)), ("UNSUPPORTED", "dim", dict(dim=-64)),
    ("UNSUPPORTED", "dim", dict(dim=60)), ("UNSUPPORTED", "dim", dict(dim=8200)), ("UNSUPPORTED", "dtype", dict(dtype=-1)), ("ARG", "rms", dict(rms=2)),
    ("ARG", "gate_first must", dict(first=2)), ("ARG", "without a gate", dict(first=1)), ("ARG", "eps", dict(eps=-1.0)),
    ("ARG", "eps", dict(eps=float("nan"))), ("ARG", "x row stride", dict(st=(64, 0, 0, 0, 0))), ("ARG", "gate row stride", dict(z=4 * P, st=(128, 100, 0, 0, 0))),
    ("ARG", "out row stride", dict(st=(128, 0, 132, 0, 0))), ("ARG", "aligned", dict(x=P + 8)), ("ARG", "aligned", dict(w=P + 8)),
    ("ARG", "aligned", dict(b=P + 4)), ("ARG", "NULL", dict(x=None)), ("UNSUPPORTED", "item range", dict(rows=1 << 30, groups=4)),
    ("UNSUPPORTED", "item range", dict(rows=1, groups=1 << 20, dim=8192)),
]


@pytest.mark.parametrize("code,words,kw", NORMS + [
    ("ARG", "NULL", dict(out=None)), ("ARG", "aligned", dict(out=P + 2)), ("ARG", "in the place of x", dict(out=P, st=(128, 0, 136, 0, 0))),
    ("ARG", "in the place of gate", dict(z=2 * P, st=(128, 136, 128, 0, 0))),
])
def test_norm_refusals(gdn, code, words, kw):
    rc, msg = ln(gdn, **kw)
    assert rc == getattr(gdn, "GDN_ERR_" + code) and words in msg, msg


@pytest.mark.parametrize("code,words,kw", [(c, w, dict(k, dz=5 * P) if "z" in k else k) for c, w, k in NORMS] + [
    ("ARG", "dout row stride", dict(st=(0, 0, 0, 8, 0))), ("ARG", "dgate row stride", dict(z=4 * P, dz=5 * P, st=(0, 0, 0, 0, 8))),
    ("ARG", "NULL", dict(dout=None)), ("ARG", "NULL", dict(dx=None)), ("ARG", "NULL", dict(z=4 * P)), ("ARG", "without a gate", dict(dz=P)),
    ("ARG", "aligned", dict(dx=P + 2)), ("ARG", "smaller", dict(ws=P, size=16)), ("ARG", "256-byte", dict(ws=P + 16, size=1 << 30)),
    ("ARG", "the same", dict(z=4 * P, dz=3 * P)), ("ARG", "in the place of dout", dict(dx=2 * P, st=(0, 0, 136, 0, 0))),
])
def test_norm_backward_refusals(gdn, code, words, kw):
    rc, msg = ln_back(gdn, **kw)
    assert rc == getattr(gdn, "GDN_ERR_" + code) and words in msg, msg


def test_empty_calls(gdn):
    none = dict(x=None, out=None)
    assert conv(gdn, T=0, **none)[0] == conv(gdn, B=0, **none)[0] == gdn.GDN_OK
    assert conv_back(gdn, T=0, x=None, dout=None, dx=None, dw=None, db=None, dh0=None)[0] == gdn.GDN_OK
    nothing = dict(q=None, k=None, v=None, dt=None, a=None, state=None, out=None)
    assert ssm(gdn, T=0, **nothing)[0] == step(gdn, B=0, **nothing)[0] == gdn.GDN_OK
    assert ln(gdn, rows=0, **none)[0] == ln_back(gdn, rows=0, x=None, dout=None, dx=None, dw=None, db=None)[0] == gdn.GDN_OK
    assert gdn.last_launch_count() == 0
    lib = gdn.load()
    assert lib.gdn_causal_conv_backward_workspace_bytes(0, 64, 4) == lib.gdn_causal_conv_backward_workspace_bytes(9, 60, 4) == 0
    assert lib.gdn_layer_norm_backward_workspace_bytes(0, 1, 64) == lib.gdn_layer_norm_backward_workspace_bytes(9, 1, 60) == 0
    for bad in ((0, 9, 1, 2, 128, 64, 0), (1, 9, 0, 2, 128, 64, 0), (1, 9, 2, 3, 128, 64, 0), (1, 9, 1, 2, 96, 64, 0)):
        assert lib.gdn_ssm_scan_workspace_bytes(*bad) == 0


# ---- the binding --------------------------------------------------------------------------

def t(*shape, dtype="bfloat16", card=0):
    return OnCard(*shape, dtype=dtype, card=card)


def f32(*shape):
    return t(*shape, dtype="float32")


CONV = dict(x=(6, 64), weight=(64, 4, "float32"), out=(6, 64), bias=(64, "float32"), state=(2, 3, 64), cu_seqlens=(3, "int32"))
CONV_BACK = dict(x=(6, 64), weight=(64, 4, "float32"), dout=(6, 64), dx=(6, 64), dweight=(64, 4, "float32"), dbias=(64, "float32"), bias=(64, "float32"),
                 h0=(2, 3, 64), dST=(2, 3, 64), dh0=(2, 3, 64), cu_seqlens=(3, "int32"), workspace=(1 << 20, "uint8"))
STEP = dict(q=(2, 128), k=(2, 128), v=(2, 128), dt=(2, 2, "float32"), a=(2, "float32"), state=(2, 2, 128, 64, "float32"), out=(2, 128), dt_bias=(2, "float32"),
            skip=(2, "float32"))
SCAN = dict(STEP, cu_seqlens=(3, "int32"), workspace=(1 << 20, "uint8"))
NORM = dict(x=(6, 128), out=(6, 128), weight=(64, "float32"), bias=(64, "float32"), gate=(6, 128))
NORM_BACK = dict(x=(6, 128), dout=(6, 128), dx=(6, 128), dweight=(64, "float32"), dbias=(64, "float32"), weight=(64, "float32"), bias=(64, "float32"),
                 gate=(6, 128), dgate=(6, 128), workspace=(1 << 20, "uint8"))
SIZES = dict(nk=1, nv=2, dk=128, dv=64)
CALLS = [("causal_conv", CONV, {}), ("causal_conv_backward", CONV_BACK, {}), ("ssm_scan", SCAN, SIZES), ("ssm_decode", STEP, SIZES),
         ("layer_norm", NORM, dict(dim=64)), ("layer_norm_backward", NORM_BACK, dict(dim=64))]


def make(spec, **cards):
    return {n: t(*(x for x in s if not isinstance(x, str)), dtype=s[-1] if isinstance(s[-1], str) else "bfloat16", card=cards.get(n, cards.get("all", 0)))
            for n, s in spec.items()}


@pytest.mark.parametrize("name,tensors,kw", CALLS, ids=[c[0] for c in CALLS])
def test_tensors_on_another_card(gdn, monkeypatch, name, tensors, kw):
    import torch

    gdn._setup()
    monkeypatch.setattr(gdn, "_cards", 2)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    for n in tensors:
        refused(gdn, lambda: getattr(gdn, name)(**make(tensors, **{n: 1}), **kw, stream=0), f"{n} is on")
        refused(gdn, lambda: getattr(gdn, name)(**make(tensors, **{n: -1}), **kw, stream=0), f"{n} is on")
    refused(gdn, lambda: getattr(gdn, name)(**make(tensors, all=1), **kw, stream=0), "the current device is cuda:0")


@pytest.mark.parametrize("name,tensors,kw", CALLS, ids=[c[0] for c in CALLS])
def test_host_tensors_types_and_sizes(gdn, name, tensors, kw):
    """Each tensor by itself as a host tensor, of another type, and of another size."""
    import torch

    for n, s in tensors.items():
        shape, dtype = [x for x in s if not isinstance(x, str)], s[-1] if isinstance(s[-1], str) else "bfloat16"
        bad = [("is_cuda", torch.empty(*shape, dtype=getattr(torch, dtype), device="meta"))]
        if n != "workspace":
            bad.append(("type", t(*shape, dtype="float64")))
            if n != "cu_seqlens":
                bad.append(("size", t(*shape[:-1], shape[-1] + 8, dtype=dtype)))
        for what, tensor in bad:
            args = make(tensors)
            args[n] = tensor
            with pytest.raises(gdn.GdnError) as e:
                getattr(gdn, name)(**args, **kw, stream=0)
            assert e.value.code == gdn.GDN_ERR_ARG, (n, what)


def test_batches(gdn):
    a = make(CONV)
    cu = a.pop("cu_seqlens")
    refused(gdn, lambda: gdn.causal_conv(**a, stream=0), "dense batches need B and T")
    refused(gdn, lambda: gdn.causal_conv(**a, B=2, stream=0), "dense batches need B and T")
    refused(gdn, lambda: gdn.causal_conv(**a, B=2, T=4, stream=0), "6 rows are not B = 2 sequences of T = 4")
    refused(gdn, lambda: gdn.causal_conv(**a, B=-2, T=-3, stream=0), "not B = -2")
    refused(gdn, lambda: gdn.causal_conv(**a, B=2, T=3, cu_seqlens=cu, stream=0), "packed ones")
    refused(gdn, lambda: gdn.causal_conv(**a, cu_seqlens=t(0, dtype="int32"), stream=0), "one element")
    refused(gdn, lambda: gdn.causal_conv(**dict(a, state=t(3, 3, 64)), cu_seqlens=cu, stream=0), "[2, 3, 64]")
    refused(gdn, lambda: gdn.causal_conv(**dict(a, state=t(2, dtype="int32")), cu_seqlens=cu, state_is_table=True, stream=0), "table")
    refused(gdn, lambda: gdn.causal_conv(**dict(a, weight=f32(256)), cu_seqlens=cu, stream=0), "[channels, width]")
    s = make(SCAN)
    s.pop("cu_seqlens")
    refused(gdn, lambda: gdn.ssm_scan(**s, **SIZES, B=1, T=3, stream=0), "2 rows are not")


def test_rows_over_one_another(gdn):
    """expand() gives rows without a stride, which the library would take for packed ones."""
    one = t(1, 64)
    one.layout = one.layout.expand(6, 64)
    a = make(CONV)
    refused(gdn, lambda: gdn.causal_conv(**dict(a, x=one), stream=0), "row stride")
    refused(gdn, lambda: gdn.causal_conv(**dict(a, out=one), stream=0), "row stride")
    wide = t(1, 128)
    wide.layout = wide.layout.expand(6, 128)
    refused(gdn, lambda: gdn.layer_norm(wide, t(6, 128), dim=64, stream=0), "row stride")
    refused(gdn, lambda: gdn.layer_norm(t(6, 128), t(6, 128), dim=48, stream=0), "groups of 48")
    refused(gdn, lambda: gdn.layer_norm(t(6, 128), t(6, 128), dim=0, stream=0), "dim")
    refused(gdn, lambda: gdn.layer_norm(t(128), t(128), dim=64, stream=0), "rows")


def test_step_refuses_what_other_heads_read_as_output(gdn):
    for name in ("q", "k"):
        rc, msg = step(gdn, **{name: 2 * P})
        assert rc == gdn.GDN_ERR_ARG and "must not be q or k" in msg, msg
    rc, msg = step(gdn, v=2 * P, o=opt(4, 512))
    assert rc == gdn.GDN_ERR_ARG and "in the place of v" in msg, msg


def test_tables_of_no_sequences(gdn):
    """An empty tensor's address is 0, also that of an empty table: a batch of no sequences has nothing to refuse."""
    assert conv(gdn, B=0, x=None, out=None, state=None, table=1)[0] == gdn.GDN_OK
    rows = t(0, 64)
    for kw in (dict(B=0, T=3), dict(cu_seqlens=t(1, dtype="int32"))):
        gdn.causal_conv(rows, f32(64, 4), t(0, 64), state=t(0, dtype="int64"), state_is_table=True, stream=0, **kw)
    step = dict(q=t(0, 128), k=t(0, 128), v=t(0, 128), dt=f32(0, 2), a=f32(2), state=t(0, dtype="int64"), out=t(0, 128), state_is_table=True, stream=0, **SIZES)
    gdn.ssm_decode(**step)
    gdn.ssm_scan(**step, B=0, T=3)
