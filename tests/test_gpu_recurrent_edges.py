"""The scan's chunks at the ends of its forms, outputs of refused sequences, and norms in place, against 64 bits."""
import pytest
import torch

from tests import recurrent_reference as ref
from tests.test_gpu_recurrent import DEV, batch, check_scan, gdn, make_conv, make_norm, near, offsets, rand, ssm, ssm_want  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dk,dv,nk,nv", [(128, 64, 1, 4), (64, 64, 2, 6), (128, 128, 1, 2), (128, 64, 1, 3)])
def test_scan_partial_chunks_of_wide_decay(gdn, dk, dv, nk, nv):
    """Last chunks of 1 to 127 tokens that decay fast, behind chunks that do and that do not, in one head of a pair or both, with NaN in
    the rows behind each batch: what lies behind a sequence reaches nothing, and the chunk's own rows are all there."""
    tails = (1, 31, 77, 127)
    lens = [128 * chunks + tail for chunks in (0, 1, 2, 3, 4) for tail in tails]
    for turn, heads in enumerate((slice(None), slice(0, 1), slice(nv - 1, nv))):
        s = ssm(lens, nk, nv, dk, dv, seed=61 + turn, steps=0.02, rate=4.0)
        s["a"][heads] = -4.0
        first = 0
        for i, n in enumerate(lens):
            for c in range((n + 127) // 128):  # each sequence with its own order of the two; the last chunk is always wide
                rows = slice(first + 128 * c, first + min(128 * (c + 1), n))
                if c == n // 128 or (0x5A3C96 >> (i + 3 * c)) & 1:
                    s["dt"][rows, heads] += 400.0 / (rows.stop - rows.start)
            first += n
        z = s["dt"].double() + s["bias"].double()
        s["d"] = torch.nn.functional.softplus(z, threshold=1e4)
        want, rows = ssm_want(s, lens), sum(lens)
        bad = {n: torch.cat([s[n], torch.full((130, s[n].shape[1]), float("nan"), dtype=s[n].dtype, device=DEV)]) for n in ("q", "k", "v", "dt")}
        out, state = torch.full((rows + 130, nv * dv), 7.0, dtype=torch.bfloat16, device=DEV), s["state"].clone()
        gdn.ssm_scan(bad["q"], bad["k"], bad["v"], bad["dt"], s["a"], state, out, **s["args"], **batch(lens, True))
        gdn.check()
        check_scan(out[:rows], state, want, rows)
        assert (out[rows:] == 7).all()
        for i in (3, 18, 19):  # and alone, where NaN stands right behind it
            a, b = offsets(lens)[i], offsets(lens)[i + 1]
            one = {n: torch.cat([s[n][a:b], bad[n][rows:]]) for n in bad}
            o, S = torch.full((b - a + 130, nv * dv), 7.0, dtype=torch.bfloat16, device=DEV), s["state"][i:i + 1].clone()
            gdn.ssm_scan(one["q"], one["k"], one["v"], one["dt"], s["a"], S, o, **s["args"], **batch([b - a], True))
            gdn.check()
            assert torch.equal(o[:b - a], out[a:b]) and torch.equal(S[0], state[i]) and (o[b - a:] == 7).all()


@pytest.mark.parametrize("size", [2.0 ** -20, 1e-3, 1.0, 1e2, 1e3])
@pytest.mark.parametrize("dk,dv", [(128, 64), (128, 128), (64, 64)])
def test_scan_of_large_and_small_values(gdn, dk, dv, size):
    """Heads whose chunks decay by 60 to 141 nats, with q, k and v of any size that the header names: finite, and within the bounds of
    values about one."""
    nats = [60.0, 79.0, 81.0, 99.0, 101.0, 120.0, 139.0, 141.0]
    nv, T = len(nats), 300
    s = ssm([T], 1, nv, dk, dv, seed=71, softplus=False)
    s["args"]["dt_bias"] = None
    for n in ("q", "k", "v"):
        s[n] = (s[n].float() * size).to(torch.bfloat16)
    s["state"] *= size * size
    s["dt"] = torch.ones(T, nv, device=DEV)
    s["a"] = -torch.tensor(nats, device=DEV) / 128
    s["d"] = s["dt"].double()
    o, S, mags, M = ssm_want(s, [T])
    out, state = torch.empty(T, nv * dv, dtype=torch.bfloat16, device=DEV), s["state"].clone()
    gdn.ssm_scan(s["q"], s["k"], s["v"], s["dt"], s["a"], state, out, B=1, T=T, **s["args"])
    gdn.check()
    got = out.view(o.shape).double()
    assert torch.isfinite(got).all() and torch.isfinite(state).all()
    # the bounds of check_scan, per head: bf16 operands 2^-6 of the terms, the output 2^-8, the state 2^-14 of its terms
    near(got, o, 2.0 ** -6 * mags + 2.0 ** -8 * o.abs(), "out")
    near(state, S, 2.0 ** -14 * M, "state")
    off, term = ((got - o) ** 2).sum((0, 2)).sqrt(), (mags ** 2).sum((0, 2)).sqrt()
    assert (off <= 5e-3 * term).all(), (off / term).tolist()
    off, term = ((state.double() - S) ** 2).sum((0, 2, 3)).sqrt(), (M ** 2).sum((0, 2, 3)).sqrt()
    assert (off <= 1e-5 * term).all(), (off / term).tolist()


def test_scan_of_equal_large_values(gdn):
    """All values alike, the largest sums: 100 in every place of q, k and v, steps of 1, chunks of 139.5 nats."""
    T = 256
    full = lambda w: torch.full((T, w), 100.0, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    dt, a, state = torch.ones(T, 1, device=DEV), torch.full((1,), -1.09, device=DEV), torch.zeros(1, 1, 128, 64, device=DEV)
    out = torch.empty(T, 64, dtype=torch.bfloat16, device=DEV)
    gdn.ssm_scan(full(128), full(128), full(64), dt, a, state, out, nk=1, nv=1, dv=64, softplus=False, B=1, T=T)
    gdn.check()
    t = torch.arange(T, device=DEV, dtype=torch.float64)
    sums = (1 - torch.exp(a.double() * (t + 1))) / (1 - torch.exp(a.double()))
    near(out, (128e6 * sums)[:, None].expand(-1, 64), (2.0 ** -6 * 128e6 * sums)[:, None], "out")
    near(state, (1e4 * sums[-1]).expand_as(state), 2.0 ** -14 * 1e4 * sums[-1], "state")


BAD = [[0, 50, 40, 90], [5, 40, 60, 90], [0, 200, 60, 90], [-4, 40, 60, 90], [0, 40, 60, 200], [0, 2 ** 31 - 1, 60, 90], [0, 95, 33, 90]]


@pytest.mark.parametrize("cu", BAD)
def test_sequences_with_bad_offsets_write_nothing(gdn, cu):
    """Beside the report: rows that only refused sequences would own keep what they held, as do the rows around the buffers and the states of
    those sequences; the rows of a sequence whose offsets are its own come out as in a batch of their own."""
    rows, D, pad = 90, 64, 4
    off = torch.tensor(cu, dtype=torch.int32, device=DEV)
    held = [i for i in range(3) if 0 <= cu[i] <= cu[i + 1] <= rows]
    owners = [[i for i in held if cu[i] <= r < cu[i + 1]] for r in range(rows)]
    free = torch.tensor([not o for o in owners], device=DEV)
    s, c = ssm([30] * 3, 1, 2, 128, 64, seed=81), make_conv([30] * 3, D, 4, torch.bfloat16, seed=81)

    def framed(width):
        t = torch.full((rows + 2 * pad, width), 7.0, dtype=torch.bfloat16, device=DEV)
        return t, t[pad:-pad]

    def reported():
        with pytest.raises(gdn.GdnError) as e:
            gdn.check()
        assert e.value.code == gdn.GDN_ERR_DEVICE_STATUS

    def untouched(frame, part):
        assert (frame[:pad] == 7).all() and (frame[-pad:] == 7).all() and (part[free] == 7).all()

    def alone(i):  # a sequence's rows, and which of them no other sequence writes too
        a, b = cu[i], cu[i + 1]
        return slice(a, b), torch.tensor([owners[r] == [i] for r in range(a, b)], dtype=torch.bool, device=DEV)

    frame, out = framed(128)
    state = s["state"].clone()
    gdn.ssm_scan(s["q"], s["k"], s["v"], s["dt"], s["a"], state, out, cu_seqlens=off, **s["args"])
    reported()
    untouched(frame, out)
    for i in range(3):
        if i not in held:
            assert torch.equal(state[i], s["state"][i])
        elif cu[i] < cu[i + 1]:
            r, own = alone(i)
            one, S = torch.empty_like(out[r]), s["state"][i:i + 1].clone()
            gdn.ssm_scan(s["q"][r], s["k"][r], s["v"][r], s["dt"][r], s["a"], S, one, B=1, T=one.shape[0], **s["args"])
            assert torch.equal(one[own], out[r][own]) and torch.equal(S[0], state[i])

    frame, out = framed(D)
    state = c["h0"].clone()
    gdn.causal_conv(c["x"], c["w"], out, bias=c["b"], state=state, cu_seqlens=off)
    reported()
    untouched(frame, out)
    for i in range(3):
        if i not in held:
            assert torch.equal(state[i], c["h0"][i])
        elif cu[i] < cu[i + 1]:
            r, own = alone(i)
            one, S = torch.empty_like(out[r]), c["h0"][i:i + 1].clone()
            gdn.causal_conv(c["x"][r], c["w"], one, bias=c["b"], state=S, B=1, T=one.shape[0])
            assert torch.equal(one[own], out[r][own]) and torch.equal(S[0], state[i])

    frame, dx = framed(D)
    dh0 = torch.full_like(c["h0"], 7)
    dw = torch.empty_like(c["w"])
    gdn.causal_conv_backward(c["x"], c["w"], c["dout"], dx, dw, bias=c["b"], h0=c["h0"], dST=c["dST"], dh0=dh0, cu_seqlens=off)
    reported()
    untouched(frame, dx)
    for i in range(3):
        if i not in held:
            assert (dh0[i] == 7).all()
        elif cu[i] < cu[i + 1]:
            r, own = alone(i)
            one, S = torch.empty_like(dx[r]), torch.empty_like(dh0[i:i + 1])
            gdn.causal_conv_backward(c["x"][r], c["w"], c["dout"][r], one, bias=c["b"], h0=c["h0"][i:i + 1], dST=c["dST"][i:i + 1], dh0=S, B=1, T=one.shape[0])
            assert torch.equal(one[own], dx[r][own]) and torch.equal(S[0], dh0[i])
    gdn.check()


@pytest.mark.parametrize("gate,first,kind", [(False, False, "layer"), (True, False, "rms"), (True, True, "layer")])
@pytest.mark.parametrize("dim,dtype", [(256, torch.bfloat16), (1000, torch.bfloat16), (1024, torch.float32), (4096, torch.float16), (8192, torch.bfloat16), (8192, torch.float32)])
def test_wide_norms_in_place(gdn, dim, dtype, gate, first, kind):
    """Rows that the backward has under way while it writes others: several a CTA, outputs in the place of each input that they may take."""
    c = make_norm(2000, 1, dim, dtype, 0, kind, "before" if first else "after" if gate else None, seed=91)
    f = c["form"]
    want = torch.empty_like(c["x"])
    gdn.layer_norm(c["x"], want, weight=c["weight"], bias=c["bias"], gate=c["gate"], **f)
    places = ["x", "gate"] if gate else ["x"]
    for place in places:
        t = {n: c[n].clone() for n in places}
        gdn.layer_norm(t["x"], t[place], weight=c["weight"], bias=c["bias"], gate=t.get("gate"), **f)
        assert torch.equal(t[place], want), place
    new = lambda t: torch.empty_like(t)  # noqa: E731
    dx, dz, dw, db = new(c["x"]), new(c["x"]) if gate else None, new(c["weight"]), new(c["bias"])
    gdn.layer_norm_backward(c["x"], c["dout"], dx, dw, db, weight=c["weight"], bias=c["bias"], gate=c["gate"], dgate=dz, **f)
    inputs = ["x", "dout"] + (["gate"] if gate else [])
    for a in inputs:
        for b in inputs if gate else [None]:
            if a == b:
                continue
            t = {n: c[n].clone() for n in inputs}
            w, d = new(dw), new(db)
            gdn.layer_norm_backward(t["x"], t["dout"], t[a], w, d, weight=c["weight"], bias=c["bias"], gate=t.get("gate"), dgate=t[b] if gate else None, **f)
            assert torch.equal(t[a], dx) and torch.equal(w, dw) and torch.equal(d, db) and (not gate or torch.equal(t[b], dz)), (a, b)
    gdn.check()


@pytest.mark.parametrize("B,nk,nv,dk,dv,pad", [(3, 1, 24, 128, 64, 8), (17, 4, 4, 128, 128, 0), (300, 2, 6, 64, 64, 16)])
def test_step_in_the_place_of_v(gdn, B, nk, nv, dk, dv, pad):
    s = ssm([1] * B, nk, nv, dk, dv, pad, steps=0.5, seed=95)
    out, states = torch.empty(B, nv * dv, dtype=torch.bfloat16, device=DEV), [s["state"].clone() for _ in range(2)]
    gdn.ssm_decode(s["q"], s["k"], s["v"], s["dt"], s["a"], states[0], out, **s["args"])
    gdn.ssm_decode(s["q"], s["k"], s["v"], s["dt"], s["a"], states[1], s["v"], **s["args"])
    gdn.check()
    assert torch.equal(out, s["v"]) and torch.equal(*states)


@pytest.mark.parametrize("dk,dv,nk,nv", [(128, 64, 1, 4), (128, 128, 1, 2), (64, 64, 1, 3)])
def test_scan_of_tokens_without_a_step(gdn, dk, dv, nk, nv):
    """Steps of exactly zero (dt of -infinity under softplus, as masked tokens have it): such a token leaves the state alone, in chunks of
    either kind, at their ends, and for whole chunks and sequences."""
    lens = [300, 128, 40, 129]
    s = ssm(lens, nk, nv, dk, dv, seed=97, steps=0.05, rate=8.0)
    low, rows = float("-inf"), sum(lens)
    s["a"][0] = -16.0
    s["dt"][:300, 0] += 2.0  # a head whose chunks decay by much
    for r in (slice(0, 3), slice(17, 20), slice(96, 160), slice(255, 257), slice(290, 300), slice(300, 428), slice(430, 468), slice(469, 470), slice(596, 597)):
        s["dt"][r] = low
    s["dt"][130:140, 1:] = low
    s["d"] = torch.nn.functional.softplus(s["dt"].double() + s["bias"].double(), threshold=1e4)
    assert (s["d"][300:428] == 0).all()
    o, S, mags, M = ssm_want(s, lens)
    out, state = torch.empty(rows, nv * dv, dtype=torch.bfloat16, device=DEV), s["state"].clone()
    gdn.ssm_scan(s["q"], s["k"], s["v"], s["dt"], s["a"], state, out, **s["args"], **batch(lens, True))
    gdn.check()
    check_scan(out, state, (o, S, mags, M), rows)
    near(state[1], s["state"][1].double(), 2.0 ** -22 * s["state"][1].double().abs(), "a sequence without steps")  # e^0 S, one rounding at most
    one = s["state"].clone()
    gdn.ssm_decode(s["q"][:4], s["k"][:4], s["v"][:4], torch.full_like(s["dt"][:4], low), s["a"], one, out[:4], **s["args"])
    gdn.check()
    assert torch.equal(one, s["state"])
