"""The softmax-attention layer of a hybrid model, as a serving program and a training step use it:

  * a prompt's keys and values go into a paged cache, normed and rotated on the way, and its queries attend,
  * a tree of drafted tokens is appended behind it and verified in one call,
  * the accepted path is kept: its tokens move up to the end of the context,
  * the next token is decoded,
  * and, for training, the gradient of the head norm with the rotation.

Prints how far the tree's rows are from decoding the same tokens one by one. Run from the repository's root:

    python examples/hybrid_attention.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import gated_delta_rule_17_gb300 as gdn  # noqa: E402


class AttentionLayer:
    """Heads, weights, rotation tables and the paged cache of one layer; every call runs on the current stream."""

    def __init__(self, nq=32, nkv=8, d=128, rot=64, pages=64, page=16, sequences=2, positions=4096, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.nq, self.nkv, self.d, self.page = nq, nkv, d, page
        self.q_weight = 1 + 0.1 * torch.randn(d, generator=g, device=device)
        self.k_weight = 1 + 0.1 * torch.randn(d, generator=g, device=device)
        angle = torch.arange(positions, device=device)[:, None] * 10000.0 ** (-torch.arange(0, rot, 2, device=device) / rot)
        self.cos, self.sin = angle.cos(), angle.sin()
        self.k_cache = torch.zeros(pages, page, nkv, d, dtype=torch.bfloat16, device=device)
        self.v_cache = torch.zeros_like(self.k_cache)
        # the pages dealt out to the sequences beforehand; a server would hand them out as they fill
        each = pages // sequences
        self.table = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))[:each * sequences].view(sequences, each).int().to(device)
        self.lens = torch.zeros(sequences, dtype=torch.int32, device=device)
        self.scratch = torch.empty(gdn.tree_attention_workspace_bytes(nq, nkv, d), dtype=torch.uint8, device=device)

    def attend(self, q, k, v, cu_rows, positions, max_rows, mask=None):
        """Appends the rows' keys and values behind each sequence's context and lets the rows attend."""
        q_rot = torch.empty_like(q)
        gdn.head_norm_rope(q, None, positions, self.cos, self.sin, q_rot, None, nq=self.nq, nkv=0, head_dim=self.d,
                           q_weight=self.q_weight)
        gdn.paged_append(k, v, self.k_cache, self.v_cache, self.table, self.lens, nkv=self.nkv, head_dim=self.d,
                         cu_rows=cu_rows, positions=positions, cos=self.cos, sin=self.sin, norm=True, k_weight=self.k_weight)
        out = torch.empty_like(q)
        gdn.tree_attention(q_rot, self.k_cache, self.v_cache, self.table, self.lens, out, nq=self.nq, nkv=self.nkv,
                           head_dim=self.d, cu_rows=cu_rows, mask=mask, max_rows=max_rows, workspace=self.scratch)
        return out


def tree_mask(parents):
    """parents[i]: the parent of drafted token i in its tree (-1: the context), parents first. Returns the mask words
    (each row sees itself and its ancestors) and the depths."""
    rows, depth = [], []
    for i, p in enumerate(parents):
        rows.append((1 << i) | (rows[p] if p >= 0 else 0))
        depth.append(depth[p] + 1 if p >= 0 else 0)
    words = [[((r >> (64 * w)) & (2 ** 64 - 1)) for w in range((len(parents) + 63) // 64)] for r in rows]
    signed = [[x - 2 ** 64 if x >= 2 ** 63 else x for x in r] for r in words]
    return torch.tensor(signed, dtype=torch.int64), torch.tensor(depth, dtype=torch.int32)


def project(layer, tokens, g):
    """Stands in for the layer's projections: random q, k, v rows."""
    make = lambda heads: torch.randn(tokens, heads * layer.d, generator=g, device="cuda").bfloat16()  # noqa: E731
    return make(layer.nq), make(layer.nkv), make(layer.nkv)


def verify_a_tree(prompt=(150, 70), parents=(-1, 0, 0, 1, 1, 2, 4, 4, -1, 8), accepted=(0, 1, 4, 7)):
    """Prompts, one draft tree a sequence, the accepted path kept, one more token. Returns the largest difference
    between the tree's accepted rows and the same tokens decoded one by one, relative to the rows' size."""
    layer = AttentionLayer(sequences=len(prompt))
    g = torch.Generator(device="cuda").manual_seed(1)
    B, n, dev = len(prompt), len(parents), "cuda"

    cu = torch.tensor([0] + list(torch.tensor(prompt).cumsum(0)), dtype=torch.int32, device=dev)
    at = torch.cat([torch.arange(p) for p in prompt]).int().to(dev)
    layer.attend(*project(layer, sum(prompt), g), cu, at, max(prompt))
    layer.lens += torch.tensor(prompt, dtype=torch.int32, device=dev)

    words, depth = tree_mask(parents)
    cu = torch.arange(0, B * n + 1, n, dtype=torch.int32, device=dev)
    at = (layer.lens[:, None] + depth.to(dev)).flatten().int()
    q, k, v = project(layer, B * n, g)
    tree = layer.attend(q, k, v, cu, at, n, words.repeat(B, 1).to(dev))

    # the accepted tokens again, one by one, at the end of the context: the plain decode of the same path, which
    # leaves the cache as if nothing else had been drafted
    worst = 0.0
    for i in accepted:
        rows = torch.arange(B, device=dev) * n + i
        one = layer.attend(q[rows], k[rows], v[rows], None, layer.lens.clone(), 1)
        worst = max(worst, float((one.float() - tree[rows].float()).norm() / one.float().norm()))
        layer.lens += 1
    layer.attend(*project(layer, B, g), None, layer.lens.clone(), 1)
    gdn.check()
    return worst


def train_the_norm(rows=512, nq=32, nkv=8, d=128):
    """One gradient step on the norms' weights for a random target; returns the loss before and after."""
    layer = AttentionLayer(nq=nq, nkv=nkv, d=d)
    g = torch.Generator(device="cuda").manual_seed(2)
    q, k, _ = project(layer, rows, g)
    want_q, want_k, _ = project(layer, rows, g)
    at = torch.arange(rows, dtype=torch.int32, device="cuda")
    kw = dict(nq=nq, nkv=nkv, head_dim=d, q_weight=layer.q_weight, k_weight=layer.k_weight)

    def forward():
        yq, yk = torch.empty_like(q), torch.empty_like(k)
        gdn.head_norm_rope(q, k, at, layer.cos, layer.sin, yq, yk, **kw)
        return yq, yk

    def loss(yq, yk):
        return float(((yq.float() - want_q.float()) ** 2).mean() + ((yk.float() - want_k.float()) ** 2).mean())

    yq, yk = forward()
    before = loss(yq, yk)
    gq, gk = (2 * (yq.float() - want_q.float()) / yq.numel()).bfloat16(), (2 * (yk.float() - want_k.float()) / yk.numel()).bfloat16()
    dq, dk = torch.empty_like(q), torch.empty_like(k)
    dqw, dkw = torch.empty_like(layer.q_weight), torch.empty_like(layer.k_weight)
    gdn.head_norm_rope_backward(q, k, at, layer.cos, layer.sin, gq, gk, dq, dk, dqw, dkw, **kw)
    layer.q_weight -= 20.0 * dqw
    layer.k_weight -= 20.0 * dkw
    after = loss(*forward())
    gdn.check()
    return before, after


if __name__ == "__main__":
    from gated_delta_rule_17_gb300 import build

    build.build()
    print(f"tree rows against one-by-one decoding: {verify_a_tree():.2e} of their size")
    before, after = train_the_norm()
    print(f"a step on the norms' weights: loss {before:.4f} -> {after:.4f}")
