"""Calls that the softmax-attention entry points have to refuse, by name and before anything is launched. No GPU."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def gdn():
    from gated_delta_rule_17_gb300 import build

    build.build()
    import gated_delta_rule_17_gb300 as gdn

    gdn.load()
    return gdn


# Run by a process of its own: what is refused here once ended the process (a division by zero).
HEAD_SIZE = """
import ctypes
import gated_delta_rule_17_gb300 as gdn
lib, P, d = gdn.load(), 256, {d}
cache = gdn.Paged(P, P, 4096, 256, 128, 4096, 256, 128, 9, 16, P, 4, 4, 3, 5, P, P)
at = ctypes.addressof(cache)
calls = dict(
    head_norm_rope=lambda: lib.gdn_head_norm_rope(P, P, P, None, None, None, 1e-6, P, P, 4, 4, 2, d, 0, None, None),
    head_norm_rope_backward=lambda: lib.gdn_head_norm_rope_backward(P, P, P, None, None, None, 1e-6, P, P, P, P, P, P, 4, 4, 2, d, 0,
                                                                    None, None, 0, None),
    paged_append=lambda: lib.gdn_paged_append(P, P, at, None, None, 0, None, 1e-6, 2, d, 0, 0, 0, None),
    tree_attention=lambda: lib.gdn_tree_attention(P, at, None, 0, 0.1, P, 4, 2, d, 0, 0, 0, 0, None, 0, None))
for name, call in calls.items():
    rc = call()
    assert rc == gdn.GDN_ERR_UNSUPPORTED and b"head_dim" in lib.gdn_last_error(), (name, rc, lib.gdn_last_error())
assert lib.gdn_head_norm_rope_backward_workspace_bytes(4, 4, 2, d) == 0 and lib.gdn_tree_attention_workspace_bytes(4, 2, d) == 0
"""


@pytest.mark.parametrize("d", [0, -1, -128, 96, 1 << 30])
def test_head_sizes(gdn, d):
    r = subprocess.run([sys.executable, "-c", HEAD_SIZE.format(d=d)], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])


class OnCard:
    """A tensor's layout with an address that nothing may follow, as if it lay on a card: what is tested is refused
    before it is read."""

    is_cuda = True

    def __init__(self, *shape, dtype="bfloat16", card=0):
        import torch

        self.layout, self.card = torch.empty(*shape, dtype=getattr(torch, dtype), device="meta"), card

    def get_device(self):
        return self.card

    def data_ptr(self):
        return 256 if self.layout.numel() else 0

    def __getattr__(self, name):
        return getattr(self.layout, name)


def refused(gdn, call, words):
    with pytest.raises(gdn.GdnError) as e:
        call()
    assert e.value.code in (gdn.GDN_ERR_ARG, gdn.GDN_ERR_UNSUPPORTED) and words in str(e.value), str(e.value)


def attend(gdn, rows=4, d=128, **kw):
    a = dict(q=OnCard(rows, 4 * d), k_cache=OnCard(3, 16, 2, d), v_cache=OnCard(3, 16, 2, d), block_table=OnCard(rows, 2, dtype="int32"),
             ctx_lens=OnCard(rows, dtype="int32"), out=OnCard(rows, 4 * d), nq=4, nkv=2, head_dim=d, stream=0)
    a.update(kw)
    return gdn.tree_attention(**a)


def test_attention_over_heads_of_nothing(gdn):
    refused(gdn, lambda: attend(gdn, d=0), "head_dim")


def test_a_mask_of_no_words_is_not_no_mask(gdn):
    # such a tensor has no address, which the library would take for "each row sees those up to itself"
    refused(gdn, lambda: attend(gdn, mask=OnCard(4, 0, dtype="int64")), "word")
    attend(gdn, rows=0, mask=OnCard(0, 0, dtype="int64"))  # no rows: nothing to see, with or without words
    attend(gdn, rows=0, mask=OnCard(0, 2, dtype="int64"))
    assert gdn.last_launch_count() == 0


def norm(gdn, q, q_out=None, **kw):
    return gdn.head_norm_rope(q, None, None, None, None, q_out if q_out is not None else q, None, nq=2, nkv=0, stream=0, **kw)


def test_rows_that_hold_more_than_the_heads(gdn):
    # a batch of sequences in place of their rows: only the first token of each would be worked on
    batch, grad = OnCard(2, 5, 256), OnCard(2, 5, 256, dtype="float32")
    refused(gdn, lambda: norm(gdn, batch), "elements")
    refused(gdn, lambda: norm(gdn, OnCard(2, 256), batch), "elements")
    refused(gdn, lambda: gdn.head_norm_rope_backward(grad, None, None, None, None, grad, None, grad, None, nq=2, nkv=0, stream=0), "elements")
    kc, table, lens = OnCard(3, 16, 2, 128), OnCard(2, 2, dtype="int32"), OnCard(2, dtype="int32")
    refused(gdn, lambda: gdn.paged_append(batch, batch, kc, kc, table, lens, nkv=2, stream=0), "elements")
    refused(gdn, lambda: gdn.paged_append(OnCard(2, 256), batch, kc, kc, table, lens, nkv=2, stream=0), "elements")
    refused(gdn, lambda: attend(gdn, rows=2, q=OnCard(2, 5, 4 * 128)), "elements")
    refused(gdn, lambda: attend(gdn, rows=2, out=OnCard(2, 5, 4 * 128)), "elements")
    # and a row with more heads than are worked on, in place of a slice of it
    refused(gdn, lambda: norm(gdn, OnCard(4, 3, 128)), "elements")
    refused(gdn, lambda: norm(gdn, OnCard(4, 1, 128)), "elements")
    refused(gdn, lambda: norm(gdn, OnCard(4 * 256)), "2-D")


NORM = dict(q=(4, 256), k=(4, 128), positions=(4, "int32"), cos=(9, 64, "float32"), sin=(9, 64, "float32"), q_out=(4, 256),
            k_out=(4, 128), q_weight=(128, "float32"), k_weight=(128, "float32"))
BACK = {n: s for n, s in NORM.items() if not n.endswith("_out")}
BACK.update(q_grad=(4, 256), k_grad=(4, 128), dq=(4, 256), dk=(4, 128), dq_weight=(128, "float32"), dk_weight=(128, "float32"),
            workspace=(1 << 24, "uint8"))
CACHE = dict(k_cache=(3, 16, 1, 128), v_cache=(3, 16, 1, 128), block_table=(2, 2, "int32"), ctx_lens=(2, "int32"), cu_rows=(3, "int32"))
APPEND = dict(CACHE, k=(4, 128), v=(4, 128), positions=(4, "int32"), cos=(9, 64, "float32"), sin=(9, 64, "float32"), k_weight=(128, "float32"))
ATTEND = dict(CACHE, q=(4, 256), out=(4, 256), mask=(4, 1, "int64"), workspace=(1 << 24, "uint8"))
CALLS = [("head_norm_rope", NORM, dict(nq=2, nkv=1)), ("head_norm_rope_backward", BACK, dict(nq=2, nkv=1)),
         ("paged_append", APPEND, dict(nkv=1, norm=True)), ("tree_attention", ATTEND, dict(nq=2, nkv=1))]


@pytest.mark.parametrize("name,tensors,kw", CALLS, ids=[c[0] for c in CALLS])
def test_tensors_on_another_card(gdn, monkeypatch, name, tensors, kw):
    # the launch goes to the current card, and a kernel there cannot take another's addresses
    import torch

    gdn._setup()
    monkeypatch.setattr(gdn, "_cards", 2)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)

    def call(**cards):
        ts = {n: OnCard(*(x for x in s if not isinstance(x, str)), dtype=s[-1] if isinstance(s[-1], str) else "bfloat16",
                        card=cards.get(n, cards.get("all", 0))) for n, s in tensors.items()}
        return getattr(gdn, name)(**ts, **kw, stream=0)

    for n in tensors:
        refused(gdn, lambda: call(**{n: 1}), f"{n} is on")
        refused(gdn, lambda: call(**{n: -1}), f"{n} is on")
    refused(gdn, lambda: call(all=1), "the current device is cuda:0")
