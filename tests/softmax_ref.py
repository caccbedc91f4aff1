"""Plain float64 softmax attention on the band and rotary positions, and bounds on
what rounding may do to a kernel's results.

Half a step of a type is h = eps / 2 relative to the value (bf16 2^-8, fp32 2^-24).
With s the relative error of a probability P that is not yet rounded (below), a
kernel that rounds P and dS to the storage type for its second products, and its
results once, is off by at most
    O    h |O| + (h + s) P |V|
    D    E = |dO| . (h |O| + (h + s) P |V|)        (D = dO . O from the rounded O)
    dQ   h |dQ| + c [ (h + 2s) |P| (|dP| + |D|) + E P ] |K|
    dK   the same with the sums over queries, |Q| for |K|
    dV   h |dV| + (h + s) P^T |dO|
(absolute values inside every sum).  s: the score's fp32 product of 64 terms and its
scaling err by at most (64 + 3) 2^-24 sum |q k| c, u by as much plus the sum's n
2^-24, and the exponential by 2^-22; the tests' inputs keep sum |q k| c under 60
and n under 2^12, which gives s < 2^-11 in the worst case, and with errors of random sign
(square roots of the counts) s < 2^-15, which is used.
"""
import math

import torch

H = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
S = 2.0 ** -15
U_ATOL = 1e-5  # the row duals' absolute tolerance, as for every dual of the library


def support(B, Lq, Lk, W, causal, mask, q_pos, device):
    """[B, Lq, Lk] bool."""
    first = torch.full((B,), Lk - Lq, device=device) if q_pos is None else q_pos.long().to(device)
    p = first[:, None] + torch.arange(Lq, device=device)
    j = torch.arange(Lk, device=device)
    gap = p[:, :, None] - j
    ok = (gap <= W) & (gap >= (0 if causal else -W))
    inside = (p >= 0) & (p < Lk)
    ok &= inside[:, :, None]
    if mask is not None:
        m = mask.to(device) != 0
        ok &= m[:, None, :] & m.gather(1, p.clamp(0, Lk - 1))[:, :, None]
    return ok


def clean(x):
    return torch.nan_to_num(x.double(), nan=0.0, posinf=0.0, neginf=0.0)


def forward(q, k, v, *, W, eps=1.0, causal=False, mask=None, q_pos=None):
    """(o, u, P) in float64; non-finite inputs count as 0 (they belong to unused tokens)."""
    q, k, v = clean(q), clean(k), clean(v)
    B, Hq, Lq, d = q.shape
    G = Hq // k.shape[1]
    k, v = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    ok = support(B, Lq, k.shape[2], W, causal, mask, q_pos, q.device)[:, None]
    s = (q @ k.transpose(-1, -2) / (math.sqrt(d) * eps)).masked_fill(~ok, -math.inf)
    some = ok.any(-1).expand(s.shape[:3])
    z = torch.where(some, torch.logsumexp(s, -1), 0.0)
    P = torch.exp(s - z[..., None])
    return P @ v, -z, P


def backward(q, k, v, dO, P, *, eps=1.0):
    """(dq, dk, dv) in float64 by the formula."""
    q, k, v, dO = clean(q), clean(k), clean(v), clean(dO)
    B, Hq, Lq, d = q.shape
    Hk, Lk = k.shape[1:3]
    G, c = Hq // Hk, 1.0 / (math.sqrt(d) * eps)
    kk, vv = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    dP = dO @ vv.transpose(-1, -2)
    dS = P * (dP - (P * dP).sum(-1, keepdim=True))
    own = lambda x: x.view(B, Hk, G, Lk, d).sum(2)
    return (c * dS @ kk, own(c * dS.transpose(-1, -2) @ q), own(P.transpose(-1, -2) @ dO))


def bounds(q, k, v, dO, P, dtype, *, eps=1.0):
    """Elementwise bounds of o, dq, dk, dv (see above), the result's own rounding aside."""
    h = H[dtype]
    q, k, v = clean(q).abs(), clean(k).abs(), clean(v)
    B, Hq, Lq, d = q.shape
    Hk, Lk = k.shape[1:3]
    G, c = Hq // Hk, 1.0 / (math.sqrt(d) * eps)
    k, v = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    own = lambda x: x.view(B, Hk, G, Lk, d).sum(2)
    out = {"o": (h + S) * (P @ v.abs())}
    if dO is None:
        return out
    dO = clean(dO)
    o = P @ v
    dP = dO @ v.transpose(-1, -2)
    size = dO.abs() @ v.abs().transpose(-1, -2)  # |dP|'s terms, for its own fp32 errors
    D = (P * dP).sum(-1, keepdim=True)
    E = (dO.abs() * (h * o.abs() + out["o"])).sum(-1, keepdim=True)
    dS = P * ((h + 2 * S) * (dP.abs() + D.abs()) + 2.0 ** -18 * size + E)
    out["dq"] = c * dS @ k
    out["dk"] = own(c * dS.transpose(-1, -2) @ q)
    out["dv"] = own((h + S) * P.transpose(-1, -2) @ dO.abs())
    return out


def close(name, got, want, extra, dtype):
    """|got - want| <= h |want| + extra everywhere (1 % for the bound's own second order)."""
    got = got.double()
    assert torch.isfinite(got).all(), name
    lim = 1.01 * (H[dtype] * want.abs() + extra) + 1e-30
    over = (got - want).abs() - lim
    assert bool((over <= 0).all()), (
        name, "worst error / bound", float(((got - want).abs() / lim).max()),
        "at", (over == over.max()).nonzero()[0].tolist())


def rotate(x, freqs, pos, interleaved, scale, inverse):
    """Rotary positions of ``x`` [B,H,L,d] in float64 (``pos`` [B,L])."""
    y, n = x.double().clone(), freqs.numel()
    a = pos.double()[:, None, :, None] * freqs.double()
    c, s = scale * torch.cos(a), scale * torch.sin(a) * (-1.0 if inverse else 1.0)
    i, j = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    xa, xb = y[..., i].clone(), y[..., j].clone()
    y[..., i], y[..., j] = xa * c - xb * s, xa * s + xb * c
    return y
