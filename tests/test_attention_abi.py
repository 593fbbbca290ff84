"""Host checks of the softmax-attention entry points, without a GPU: the header's functions are exported, bad
arguments are refused by name before anything touches the device, and the binding refuses host tensors."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def gdn():
    from gated_delta_rule_17_gb300 import build

    build.build()
    import gated_delta_rule_17_gb300 as gdn

    gdn.load()
    return gdn


def test_every_declared_symbol_is_exported(gdn):
    src = open(os.path.join(ROOT, "include", "gdn_attention.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = set(re.findall(r"^\s*(?:int|size_t)\s+(gdn_[a-z_0-9]+)\s*\(", src, flags=re.M))
    assert names == {"gdn_head_norm_rope", "gdn_head_norm_rope_backward", "gdn_head_norm_rope_backward_workspace_bytes",
                     "gdn_paged_append", "gdn_tree_attention", "gdn_tree_attention_workspace_bytes"}
    for n in names:
        assert hasattr(gdn.load(), n)


P = 256  # an aligned address that no check dereferences


def at(x):
    """The address of a ctypes struct, kept alive by the caller; None for None."""
    return None if x is None else ctypes.addressof(x)


def rope(gdn, **kw):
    f = dict(cos=P, sin=P, stride=64, positions=10, rot=128, interleaved=0)
    f.update(kw)
    return gdn.Rope(*f.values())


def norm(gdn, q=P, k=P, pos=P, r=None, qw=None, kw=None, eps=1e-6, qo=P, ko=P, rows=4, nq=4, nkv=2, d=128, dtype=0, st=None):
    rc = gdn.load().gdn_head_norm_rope(q, k, pos, at(r), qw, kw, eps, qo, ko, rows, nq, nkv, d, dtype, at(st), None)
    return rc, gdn.load().gdn_last_error().decode()


@pytest.mark.parametrize("code,words,kw", [
    ("ARG", "rows", dict(rows=-1)), ("ARG", "head counts", dict(nq=0, nkv=0)), ("ARG", "head counts", dict(nq=-1)),
    ("UNSUPPORTED", "head_dim", dict(d=96)), ("UNSUPPORTED", "dtype", dict(dtype=3)), ("ARG", "eps", dict(eps=-1.0)),
    ("ARG", "eps", dict(eps=float("nan"))), ("ARG", "NULL", dict(q=None)), ("ARG", "NULL", dict(ko=None)),
    ("ARG", "aligned", dict(q=P + 8)), ("ARG", "aligned", dict(qw=P + 4)),
    ("UNSUPPORTED", "item range", dict(rows=2 ** 31 - 1)),
])
def test_norm_rope_refusals(gdn, code, words, kw):
    rc, msg = norm(gdn, **kw)
    assert rc == getattr(gdn, "GDN_ERR_" + code) and words in msg, msg


@pytest.mark.parametrize("words,kw", [
    ("rot", dict(rot=136)), ("rot", dict(rot=12)), ("rot", dict(rot=-8)), ("interleaved", dict(interleaved=2)),
    ("NULL", dict(cos=None)), ("aligned", dict(sin=P + 4)), ("positions", dict(positions=-1)), ("stride", dict(stride=60)),
    ("stride", dict(stride=66)),
])
def test_rope_refusals(gdn, words, kw):
    rc, msg = norm(gdn, r=rope(gdn, **kw))
    assert rc == gdn.GDN_ERR_ARG and words in msg, msg
    rc, msg = append(gdn, r=rope(gdn, **kw))
    assert rc == gdn.GDN_ERR_ARG and words in msg, msg


def test_norm_rope_strides_and_positions(gdn):
    assert norm(gdn, r=rope(gdn), pos=None)[0] == gdn.GDN_ERR_ARG
    for i, name in enumerate(("q ", "k ", "q_out", "k_out")):
        st = [512, 256, 512, 256, 0, 0]
        st[i] = 200
        rc, msg = norm(gdn, st=gdn.NormStrides(*st))
        assert rc == gdn.GDN_ERR_ARG and name in msg and "stride" in msg
        st[i] = 516
        assert norm(gdn, st=gdn.NormStrides(*st))[0] == gdn.GDN_ERR_ARG
    assert norm(gdn, rows=0, q=None, k=None, qo=None, ko=None)[0] == gdn.GDN_OK
    assert gdn.load().gdn_last_launch_count() == 0


def test_norm_rope_backward_refusals(gdn):
    lib = gdn.load()

    def call(gq=P, gk=P, dq=P, rows=4, st=None, ws=None, size=0, dw=P):
        rc = lib.gdn_head_norm_rope_backward(P, P, None, None, None, None, 1e-6, gq, gk, dq, P, dw, dw, rows, 4, 2, 128, 0, at(st), ws, size, None)
        return rc, lib.gdn_last_error().decode()

    for words, kw in (("gradient", dict(gq=None)), ("aligned", dict(gk=P + 2)), ("NULL", dict(dq=None)),
                      ("q_grad", dict(st=gdn.NormStrides(512, 256, 512, 256, 8, 256))),
                      ("k_grad", dict(st=gdn.NormStrides(512, 256, 512, 256, 512, 8))),
                      ("smaller", dict(ws=P, size=16)), ("256-byte", dict(ws=P + 16, size=1 << 30))):
        rc, msg = call(**kw)
        assert rc == gdn.GDN_ERR_ARG and words in msg, msg
    assert call(rows=0, gq=None, gk=None, dq=None, dw=None)[0] == gdn.GDN_OK
    assert lib.gdn_head_norm_rope_backward_workspace_bytes(0, 4, 2, 128) == 0
    assert lib.gdn_head_norm_rope_backward_workspace_bytes(10, 4, 2, 96) == 0
    assert lib.gdn_head_norm_rope_backward_workspace_bytes(10, 4, 2, 128) % 1024 == 0


def paged(gdn, **kw):
    f = dict(k=P, v=P, k_page=4096, k_token=256, k_head=128, v_page=4096, v_token=256, v_head=128, num_pages=9, page_size=16,
             block_table=P, table_stride=4, max_pages=4, B=3, rows=5, ctx_lens=P, cu_rows=P)
    f.update(kw)
    return gdn.Paged(*f.values())


def append(gdn, k=P, v=P, c=None, r=None, n=0, kw=None, eps=1e-6, nkv=2, d=128, dtype=0, ks=0, vs=0):
    lib = gdn.load()
    c = c if c is not None else paged(gdn)
    rc = lib.gdn_paged_append(k, v, at(c), None, at(r), n, kw, eps, nkv, d, dtype, ks, vs, None)
    return rc, lib.gdn_last_error().decode()


def attend(gdn, q=P, c=None, mask=None, words=0, scale=0.1, out=P, nq=4, nkv=2, d=128, dtype=0, qs=0, os_=0, most=0, ws=None, size=0):
    lib = gdn.load()
    c = c if c is not None else paged(gdn)
    rc = lib.gdn_tree_attention(q, at(c), mask, words, scale, out, nq, nkv, d, dtype, qs, os_, most, ws, size, None)
    return rc, lib.gdn_last_error().decode()


CACHE_REFUSALS = [
    ("ARG", "B = ", dict(B=-1)), ("ARG", "rows", dict(rows=-1)), ("ARG", "page_size", dict(page_size=0)),
    ("ARG", "num_pages", dict(num_pages=-1)), ("ARG", "table row stride", dict(table_stride=3)),
    ("UNSUPPORTED", "token range", dict(max_pages=1 << 28, table_stride=1 << 28)), ("ARG", "multiple of 8", dict(k_page=4100)),
    ("ARG", "multiple of 8", dict(v_token=-256)), ("ARG", "head strides", dict(v_head=64)), ("ARG", "one row a sequence", dict(cu_rows=None)),
    ("ARG", "no sequence", dict(B=0)), ("ARG", "NULL", dict(k=None)), ("ARG", "NULL", dict(block_table=None)),
    ("ARG", "NULL", dict(ctx_lens=None)), ("ARG", "aligned", dict(v=P + 8)),
]


@pytest.mark.parametrize("code,words,kw", CACHE_REFUSALS)
def test_cache_refusals(gdn, code, words, kw):
    for f in (append, attend):
        rc, msg = f(gdn, c=paged(gdn, **kw))
        assert rc == getattr(gdn, "GDN_ERR_" + code) and words in msg, msg


@pytest.mark.parametrize("code,words,kw", [
    ("ARG", "nkv", dict(nkv=0)), ("UNSUPPORTED", "head_dim", dict(d=256)), ("UNSUPPORTED", "dtype", dict(dtype=2)),
    ("ARG", "norm must", dict(n=2)), ("ARG", "without norm", dict(kw=P)), ("ARG", "eps", dict(n=1, eps=-1.0)),
    ("ARG", "k row stride", dict(ks=128)), ("ARG", "v row stride", dict(vs=260)), ("ARG", "NULL", dict(v=None)),
    ("ARG", "aligned", dict(k=P + 2)),
])
def test_append_refusals(gdn, code, words, kw):
    rc, msg = append(gdn, **kw)
    assert rc == getattr(gdn, "GDN_ERR_" + code) and words in msg, msg


@pytest.mark.parametrize("code,words,kw", [
    ("ARG", "positive", dict(nq=0)), ("UNSUPPORTED", "multiple of nkv", dict(nq=3)), ("UNSUPPORTED", "head_dim", dict(d=32)),
    ("UNSUPPORTED", "dtype", dict(dtype=2)), ("ARG", "scale", dict(scale=float("inf"))), ("ARG", "scale", dict(scale=float("nan"))),
    ("ARG", "mask_words", dict(mask=P)), ("ARG", "max_rows", dict(most=-1)), ("ARG", "q row stride", dict(qs=256)),
    ("ARG", "out row stride", dict(os_=516)), ("ARG", "NULL", dict(out=None)), ("ARG", "aligned", dict(q=P + 8)),
    ("ARG", "smaller", dict(ws=P, size=100)), ("ARG", "256-byte", dict(ws=P + 16, size=1 << 40)),
])
def test_attention_refusals(gdn, code, words, kw):
    rc, msg = attend(gdn, **kw)
    assert rc == getattr(gdn, "GDN_ERR_" + code) and words in msg, msg


def test_empty_calls(gdn):
    for f in (append, attend):
        rc, _ = f(gdn, c=paged(gdn, rows=0, k=None, v=None, block_table=None, ctx_lens=None))
        assert rc == gdn.GDN_OK and gdn.load().gdn_last_launch_count() == 0
    assert gdn.load().gdn_tree_attention_workspace_bytes(4, 2, 96) == 0
    assert gdn.load().gdn_tree_attention_workspace_bytes(4, 2, 128) <= 64 << 20


def test_binding_refuses_what_the_library_cannot_see(gdn):
    import torch

    bf, h = torch.zeros(4, 256, dtype=torch.bfloat16), torch.zeros(4, 256, dtype=torch.float64)
    cache, table, i = torch.zeros(3, 16, 2, 128, dtype=torch.bfloat16), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    calls = [
        lambda: gdn.head_norm_rope(bf, None, None, None, None, bf, None, nq=2, nkv=0),  # host tensors
        lambda: gdn.head_norm_rope(h, None, None, None, None, h, None, nq=2, nkv=0),  # type
        lambda: gdn.head_norm_rope(None, None, None, None, None, None, None, nq=0, nkv=0),
        lambda: gdn.head_norm_rope(bf, None, None, None, None, bf, None, nq=2, nkv=1),  # heads without a tensor
        lambda: gdn.head_norm_rope_backward(bf, None, None, None, None, bf, None, bf, None, nq=2, nkv=0),
        lambda: gdn.paged_append(bf, bf, cache, cache, table, i, nkv=2),
        lambda: gdn.tree_attention(bf, cache, cache, table, i, bf, nq=2, nkv=2),
        lambda: gdn.tree_attention(h, cache, cache, table, i, h, nq=2, nkv=2),
    ]
    for f in calls:
        with pytest.raises(gdn.GdnError) as e:
            f()
        assert e.value.code == gdn.GDN_ERR_ARG
    with pytest.raises(gdn.GdnError):
        gdn.paged_append(bf, bf, cache.transpose(2, 3), cache, table, i, nkv=2)


def test_packed_structs_are_the_declared_ones(gdn):
    values = list(range(1, 18))
    for cls, pack in ((gdn.Rope, gdn._ROPE), (gdn.NormStrides, gdn._STRIDES), (gdn.Paged, gdn._PAGED)):
        n = len(cls._fields_)
        raw = pack(*values[:n])
        assert len(raw) == ctypes.sizeof(cls)
        back = cls.from_buffer_copy(raw)
        assert [getattr(back, f[0]) for f in cls._fields_] == values[:n]
