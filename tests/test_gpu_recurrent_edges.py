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
