"""Plain forms in 64 bits of the operators around and beside the recurrence, with bounds on what fp32 arithmetic and the
kernels' 16-bit operands may add. u = 2^-24 is half an fp32 step; `half` half a step of the output's type."""
import torch

U = 2.0 ** -24


def half(dtype):
    return torch.finfo(dtype).eps / 2


def least(dtype):
    """Half the smallest step of the type (the rounding of results near zero)."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def conv(x, w, b, h0, cu, silu):
    """x [rows, D], h0 [B, width-1, D] or None, cu: list of offsets. Returns y (before silu), out, state, and |w||x| sums."""
    width, D = w.shape[1], w.shape[0]
    y, mags, states = x.new_zeros(x.shape), x.new_zeros(x.shape), []
    for s in range(len(cu) - 1):
        first = h0[s] if h0 is not None else x.new_zeros(width - 1, D)
        z = torch.cat([first, x[cu[s]:cu[s + 1]]])
        n = cu[s + 1] - cu[s]
        parts = [z[j:j + n] * w[:, j] for j in range(width)]
        bias = b if b is not None else 0.0
        y = torch.cat([y[:cu[s]], sum(parts) + bias, y[cu[s + 1]:]])
        mags = torch.cat([mags[:cu[s]], sum(p.abs() for p in parts) + (abs(bias) if b is not None else 0.0), mags[cu[s + 1]:]])
        states.append(z[n:])
    return y, (y * torch.sigmoid(y) if silu else y), torch.stack(states), mags


def scan(q, k, v, d, a, skip, S, cu, group):
    """q, k [rows, nk, dk], v [rows, nv, dv], d [rows, nv] steps, S [B, nv, dk, dv]. Returns out, the states after, and the same
    with every term's absolute value."""
    out, mags = torch.zeros_like(v), torch.zeros_like(v)
    S, M = S.clone(), S.abs()
    kk, qq = k.repeat_interleave(group, 1), q.repeat_interleave(group, 1)
    lens = [cu[s + 1] - cu[s] for s in range(len(cu) - 1)]
    for t in range(max(lens, default=0)):
        live = [s for s in range(len(lens)) if lens[s] > t]
        row = torch.tensor([cu[s] + t for s in live], device=v.device)
        live = torch.tensor(live, device=v.device)
        f = torch.exp(d[row] * a)[..., None, None]
        new = kk[row][..., None] * (d[row][..., None] * v[row])[..., None, :]
        S[live] = f * S[live] + new
        M[live] = f * M[live] + new.abs()
        out[row] = (qq[row][..., None] * S[live]).sum(2) + skip[:, None] * v[row]
        mags[row] = (qq[row].abs()[..., None] * M[live]).sum(2) + (skip[:, None] * v[row]).abs()
    return out, S, mags, M


def norm(x, w, b, z, gate_first, rms, eps):
    """x, z [..., dim]."""
    g = z * torch.sigmoid(z) if z is not None else None
    u = x * g if gate_first else x
    m = 0.0 if rms else u.mean(-1, keepdim=True)
    h = (u - m) / torch.sqrt(((u - m) ** 2).mean(-1, keepdim=True) + eps)
    y = h * w if w is not None else h
    if b is not None:
        y = y + b
    return y * g if z is not None and not gate_first else y
