"""Operators measured beside the Sinkhorn attention: rotary positions and banded softmax attention.

Shapes follow the rest of the repository: ``[B, H, L, 64]`` tensors, a band of
half-width ``W`` (``W >= L - 1`` is dense), a token mask ``[B, L]``, scores
``<q, k> / (sqrt(d) * eps)``, row duals ``u = -log sum_j exp(S_ij)`` (0 for a row
that attends nothing).  ``Hq`` query heads share ``Hk`` key heads in groups.
"""
import math

import torch

own = False

D = 64
BLOCK = 256  # query rows of one block of the plain form's band


# --------------------------------------------------------------------------- cases
def _rot(name, **kw):
    c = dict(name=name, op="rotary", B=1, Hq=16, Hk=16, L=1, rot=64, interleaved=False,
             scaling="none", dtype="bf16", backward=False, far=False, strided=False)
    c.update(kw)
    return c


def _att(name, **kw):
    c = dict(name=name, op="fwd", B=1, Hq=16, Hk=16, Lq=1, Lk=1, W=0, eps=1.0, causal=False,
             mask="none", ragged=False, dtype="bf16")
    c.update(kw)
    return c


def listed():
    return [
        # a batch of single tokens at far positions, as in answering: latency
        _rot("rot_token", B=16, Hq=16, Hk=4, L=1, interleaved=True, far=True),
        # queries and keys of the long-context layer, straight from a projection's [B, L, H, d]
        _rot("rot_long32k", L=32768, strided=True),
        # gradients of a padded fp32 batch, half of each head rotated
        _rot("rot_masked2k_bwd", B=4, Hq=8, Hk=8, L=2048, rot=32, interleaved=True, dtype="f32",
             backward=True),
        # gradients of the longest context, frequencies stretched for it
        _rot("rot_vjp262k_bwd", Hq=8, Hk=8, L=262144, scaling="by_parts", backward=True),
        # one new token of each of 8 sequences against caches of ragged lengths
        _att("att_token", B=8, Hq=16, Hk=4, Lq=1, Lk=32768, W=32768, causal=True, ragged=True),
        # the small parity problem, fp32
        _att("att_small512", Hq=1, Hk=1, Lq=512, Lk=512, W=64, dtype="f32"),
        # the long-context layer's band
        _att("att_long32k", Lq=32768, Lk=32768, W=256),
        # a causal layer without a band, shared key heads, an odd length
        _att("att_causal8k", Hk=4, Lq=8191, Lk=8191, W=8191, causal=True),
        # training steps (forward and backward): the small problem, latency
        _att("step_small512", op="step", Hq=1, Hk=1, Lq=512, Lk=512, W=64, dtype="f32"),
        # a padded fp32 batch
        _att("step_masked2k", op="step", B=4, Hq=8, Hk=8, Lq=2048, Lk=2048, W=128, eps=0.5,
             mask="tail", dtype="f32"),
        # the long-context layer
        _att("step_long32k", op="step", Lq=32768, Lk=32768, W=256),
        # a causal training batch with shared key heads and padding, an odd length
        _att("step_causal4k", op="step", B=2, Hk=4, Lq=4093, Lk=4093, W=4093, causal=True,
             mask="tail"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.35:
        Hk, G = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4])
        B = rng.choice([1, 2, 3, 8])
        dtype = rng.choice(["bf16", "bf16", "f32"])
        rows = 4194304 if dtype == "bf16" else 2097152  # head rows, as many as the largest case's bytes
        L = _log(rng, 1, min(262144, rows // (B * Hk * (G + 1))))
        c = _rot("", B=B, Hq=Hk * G, Hk=Hk, L=L, rot=rng.choice([16, 32, 48, 64]),
                 interleaved=rng.random() < 0.5,
                 scaling=rng.choice(["none", "linear", "ntk", "by_parts"]),
                 dtype=dtype, backward=rng.random() < 0.5,
                 far=rng.random() < 0.3, strided=rng.random() < 0.5)
    else:
        kind = rng.choice(["token", "band", "dense", "step_band", "step_dense"])
        f32 = rng.random() < 0.3
        B, Hk = rng.choice([1, 2, 4]), rng.choice([1, 2, 4])
        G = rng.choice([1, 2, 3, 4, 8])
        kw = dict(B=B, Hq=Hk * G, Hk=Hk, dtype="f32" if f32 else "bf16",
                  eps=rng.choice([0.5, 1.0, 1.0, 2.0]), causal=rng.random() < 0.5)
        pairs = 2.0e7 if f32 else 2.0e8  # (query, key) pairs over all heads
        if kind == "token":
            Lk = _log(rng, 1, 32768)
            Lq = min(Lk, rng.choice([1, 1, 1, 2, 5]))
            kw.update(Lq=Lq, Lk=Lk, W=rng.choice([Lk, Lk, max(1, Lk // 4)]), causal=True,
                      ragged=True)
        elif kind.endswith("band"):
            W = _log(rng, 1, 1024)
            L = _log(rng, 16, min(1000000 // (B * Hk * (G + 1)),
                                  max(16, int(pairs / (B * Hk * G * (2 * W + 1))))))
            kw.update(Lq=L, Lk=L, W=W, mask=rng.choice(["none", "tail", "holes"]))
        else:
            L = _log(rng, 16, int(math.sqrt(pairs / (B * Hk * G))))
            kw.update(Lq=L, Lk=L, W=L, mask=rng.choice(["none", "tail", "holes"]))
        c = _att("", op="step" if kind.startswith("step") else "fwd", **kw)
    del c["name"]
    return c


# --------------------------------------------------------------------------- inputs
def _type(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _freqs(case):
    """Radians per position of each channel pair, float64, and the factor on the result."""
    n = case["rot"] // 2
    i = torch.arange(n, dtype=torch.float64)
    base, factor, train = 10000.0, 8.0, 4096.0
    if case["scaling"] == "ntk" and n > 1:
        base = base * factor ** (n / (n - 1))
    f = base ** (-i / n)
    scale = 1.0
    if case["scaling"] == "linear":
        f = f / factor
    if case["scaling"] == "by_parts":
        # whole turns over the trained length: above 32 the pair is kept, below 1 it is
        # stretched by the factor, in between it is a mix that is linear in the index
        at = lambda turns: n * math.log(train / (turns * 2 * math.pi)) / math.log(base)
        lo, hi = max(0.0, math.floor(at(32.0))), min(n - 1.0, math.ceil(at(1.0)))
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0.0, 1.0)
        f = f / factor * ramp + f * (1 - ramp)
        scale = 0.1 * math.log(factor) + 1.0
    return f, scale


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    td, B = _type(case), case["B"]

    def randn(*s):
        return torch.randn(*s, generator=g, device="cuda").to(td)

    if case["op"] == "rotary":
        L = case["L"]
        if case["strided"]:
            q, k = (randn(B, L, case[h], D).transpose(1, 2) for h in ("Hq", "Hk"))
        else:
            q, k = (randn(B, case[h], L, D) for h in ("Hq", "Hk"))
        first = torch.zeros(B, 1, device="cuda", dtype=torch.int64)
        if case["far"]:
            first = torch.randint(0, 1 << 20, (B, 1), generator=g, device="cuda")
        pos = (first + torch.arange(L, device="cuda")).to(torch.int32)
        f, scale = _freqs(case)
        return dict(case=case, q=q, k=k, pos=pos, freqs=f.cuda(), scale=scale)
    Lq, Lk = case["Lq"], case["Lk"]
    st = dict(case=case, q=randn(B, case["Hq"], Lq, D), k=randn(B, case["Hk"], Lk, D),
              v=randn(B, case["Hk"], Lk, D), mask=None, q_pos=None)
    if case["op"] == "step":
        st["dO"] = randn(B, case["Hq"], Lq, D)
    if case["mask"] == "tail":
        n = torch.randint(Lk // 2, Lk + 1, (B, 1), generator=g, device="cuda")
        st["mask"] = (torch.arange(Lk, device="cuda")[None] < n).to(torch.uint8)
    if case["mask"] == "holes":
        st["mask"] = (torch.rand(B, Lk, generator=g, device="cuda") >= 0.1).to(torch.uint8)
    if case["ragged"]:
        # the first query's position: the caches are between half full and full
        st["q_pos"] = torch.randint(min(Lk // 2, Lk - Lq), Lk - Lq + 1, (B,), generator=g,
                                    device="cuda", dtype=torch.int32)
    return st


# --------------------------------------------------------------------------- the plain form
def _rotate(x, cos, sin, rot, interleaved):
    x = x.float()
    r, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((r, rest), -1)


def _rotary_plain(st):
    c = st["case"]
    angle = st["pos"].double()[:, None, :, None] * st["freqs"]  # [B, 1, L, rot / 2]
    cos, sin = ((f(angle) * st["scale"]).float() for f in (torch.cos, torch.sin))
    if c["backward"]:
        sin = -sin  # the rotation's transpose
    return tuple(_rotate(x, cos, sin, c["rot"], c["interleaved"]).to(x.dtype).contiguous()
                 for x in (st["q"], st["k"]))


def _band(st):
    """Keys of each block of queries: their indices ``[B, blocks, keys]`` and which
    ``[B, blocks, block, keys]`` are attended."""
    c = st["case"]
    B, Lq, Lk, W = c["B"], c["Lq"], c["Lk"], c["W"]
    right = 0 if c["causal"] else W
    dev = st["q"].device
    first = st["q_pos"].long() if st["q_pos"] is not None else torch.full((B,), Lk - Lq, device=dev)
    C = min(BLOCK, Lq)
    if c["ragged"] or C + W + right >= Lk:
        C, idx = Lq, torch.arange(Lk, device=dev).expand(B, 1, Lk)
    else:
        lo = first[:, None] + torch.arange(-(-Lq // C), device=dev) * C - W
        idx = lo[..., None] + torch.arange(C + W + right, device=dev)
    nb = idx.shape[1]
    i = torch.arange(nb * C, device=dev).view(1, nb, C, 1)
    p = first[:, None, None, None] + i
    j = idx[:, :, None, :]
    ok = (j >= 0) & (j < Lk) & (j >= p - W) & (j <= p + right) & (i < Lq)
    idx = idx.clamp(0, Lk - 1)
    if st["mask"] is not None:
        m = st["mask"].bool()
        b = torch.arange(B, device=dev)[:, None]
        ok = ok & m[b[..., None], idx][:, :, None, :]
        ok = ok & m[b, p.clamp(0, Lk - 1).view(B, -1)].view(B, nb, C, 1)
    return idx, ok, C, nb


def _blocks(x, G, nb, C):
    """[B, Hq, Lq, d] as [B, Hk, blocks, G * C, d], padded with zeros."""
    B, Hq, Lq, d = x.shape
    p = torch.zeros(B, Hq // G, G, nb * C, d, device=x.device)
    p[:, :, :, :Lq] = x.view(B, Hq // G, G, Lq, d)
    return p.view(B, Hq // G, G, nb, C, d).transpose(2, 3).reshape(B, Hq // G, nb, G * C, d)


def _unblocks(x, G, C, Lq):
    B, Hk, nb, _, d = x.shape
    x = x.view(B, Hk, nb, G, C, d).transpose(2, 3).reshape(B, Hk * G, nb * C, d)
    return x[:, :, :Lq]


def _keys(x, idx):
    """[B, Hk, Lk, d] gathered as [B, Hk, blocks, keys, d]."""
    B, Hk = x.shape[:2]
    b = torch.arange(B, device=x.device)[:, None, None, None]
    h = torch.arange(Hk, device=x.device)[:, None, None]
    return x.float()[b, h, idx[:, None]]


def _attention_plain(st):
    c = st["case"]
    G, Lq, Lk = c["Hq"] // c["Hk"], c["Lq"], c["Lk"]
    scale = 1.0 / (math.sqrt(D) * c["eps"])
    idx, ok, C, nb = _band(st)
    ok = ok[:, None, :, None].expand(-1, -1, -1, G, -1, -1).flatten(3, 4)  # [B, 1, nb, G * C, keys]
    q = _blocks(st["q"].float(), G, nb, C)
    k, v = _keys(st["k"], idx), _keys(st["v"], idx)
    s = (q @ k.transpose(-1, -2)).mul_(scale).masked_fill_(~ok, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    none = total == 0
    p = p.div_(torch.where(none, 1.0, total))
    u = torch.where(none, 0.0, -(top + torch.log(total)))
    o = p @ v
    td = st["q"].dtype
    out = dict(o=_unblocks(o, G, C, Lq).to(td).contiguous(),
               u=_unblocks(u, G, C, Lq).squeeze(-1).contiguous())
    if c["op"] == "fwd":
        return out
    dO = _blocks(st["dO"].float(), G, nb, C)
    dv = p.transpose(-1, -2) @ dO
    ds = (dO @ v.transpose(-1, -2)).sub_((dO * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    out["dq"] = _unblocks(ds @ k, G, C, Lq).to(td).contiguous()
    dk = ds.transpose(-1, -2) @ q
    at = (torch.arange(c["B"], device=idx.device)[:, None, None] * Lk + idx).flatten()

    def back(x):  # the blocks' gradients added up over the keys they share
        B, Hk = x.shape[:2]
        y = torch.zeros(Hk, B * Lk, D, device=x.device)
        y.index_add_(1, at, x.transpose(0, 1).reshape(Hk, -1, D))
        return y.view(Hk, B, Lk, D).transpose(0, 1).to(td).contiguous()

    out["dk"], out["dv"] = back(dk), back(dv)
    return out


def run(st):
    c = st["case"]
    if own:
        import banded_log_domain_b200 as sa

        if c["op"] == "rotary":
            f = sa.sinkhorn_attn_rotary_bwd if c["backward"] else sa.sinkhorn_attn_rotary_fwd
            return f(st["q"], st["k"], st["freqs"], pos=st["pos"], interleaved=c["interleaved"],
                     scale=st["scale"])
        kw = dict(W=c["W"], eps=c["eps"], causal=c["causal"], q_pos=st["q_pos"], mask=st["mask"])
        o, u = sa.sinkhorn_attn_softmax_fwd(st["q"], st["k"], st["v"], **kw)
        if c["op"] == "fwd":
            return dict(o=o, u=u)
        dq, dk, dv = sa.sinkhorn_attn_softmax_bwd(st["q"], st["k"], st["v"], o, st["dO"], u, **kw)
        return dict(o=o, u=u, dq=dq, dk=dk, dv=dv)
    return _rotary_plain(st) if c["op"] == "rotary" else _attention_plain(st)


# --------------------------------------------------------------------------- the work
def _pairs(case):
    """Attended (query, key) pairs of one head of one sequence, on average over the inputs."""
    Lq, Lk, W = case["Lq"], case["Lk"], case["W"]
    n = 0.75 * Lk if case["ragged"] or case["mask"] == "tail" else float(Lk)
    left = min(float(W), n)
    if case["ragged"]:
        return Lq * min(n, left + 1)
    rows = min(float(Lq), n)
    # rows x (left + 1) less the triangle that reaches below key 0, and the same to the right
    one = rows * left - left * left / 2 if rows >= left else rows * rows / 2
    kept = 0.81 if case["mask"] == "holes" else 1.0
    return max(rows, kept * (rows + (one if case["causal"] else 2 * one)))


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    B, Hq, Hk = case["B"], case["Hq"], case["Hk"]
    if case["op"] == "rotary":
        n = B * case["L"] * (Hq + Hk) * D
        return {"bytes": 2 * n * size + B * case["L"] * 4, "flops": 3 * n}
    Lq, Lk = case["Lq"], case["Lk"]
    kept = 0.75 * Lk if case["ragged"] else Lk
    if case["ragged"]:
        kept = min(kept, Lq + case["W"])
    q, kv = B * Hq * Lq * D * size, B * Hk * kept * D * size
    flops, moved = 4 * D * B * Hq * _pairs(case), 2 * q + 2 * kv + B * Hq * Lq * 4
    if case["op"] == "step":
        # the backward reads q, k, v, o, dO, u and writes dq, dk, dv; five products to the forward's two
        flops, moved = flops * 3.5, moved + 4 * q + 4 * kv + B * Hq * Lq * 4
    return {"bytes": moved, "flops": flops}


# --------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rotary":
        turn = torch.polar(torch.full((), st["scale"], dtype=torch.float64, device="cuda"),
                           st["pos"].double()[:, None, :, None] * st["freqs"])
        if case["backward"]:
            turn = turn.conj()
        res = []
        for x in (st["q"], st["k"]):
            y, n = x.double().clone(), case["rot"] // 2
            part = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if case["interleaved"] else \
                (slice(0, n), slice(n, 2 * n))
            z = torch.complex(y[..., part[0]], y[..., part[1]]) * turn
            y[..., part[0]], y[..., part[1]] = z.real, z.imag
            res.append(y)
        return tuple(res)
    B, Hq, Hk, Lq, Lk, W = (case[n] for n in ("B", "Hq", "Hk", "Lq", "Lk", "W"))
    dev, G, step = "cuda", Hq // Hk, case["op"] == "step"
    new = lambda *s: torch.zeros(*s, dtype=torch.float64, device=dev)
    out = dict(o=new(B, Hq, Lq, D), u=new(B, Hq, Lq))
    if step:
        out.update(dq=new(B, Hq, Lq, D), dk=new(B, Hk, Lk, D), dv=new(B, Hk, Lk, D))
    rows = 2048
    for b in range(B):
        first = int(st["q_pos"][b]) if st["q_pos"] is not None else Lk - Lq
        live = torch.ones(Lk, dtype=torch.bool, device=dev) if st["mask"] is None else st["mask"][b] > 0
        for i0 in range(0, Lq, rows):
            i1 = min(Lq, i0 + rows)
            j0 = max(0, first + i0 - W)
            j1 = min(Lk, first + i1 + (0 if case["causal"] else W))
            p = torch.arange(first + i0, first + i1, device=dev)[:, None]
            j = torch.arange(j0, j1, device=dev)[None]
            gap = p - j
            on = (gap <= W) & (gap >= (0 if case["causal"] else -W)) & live[j0:j1][None] & live[p]
            off = torch.zeros((), dtype=torch.float64, device=dev)
            bias = torch.where(on, off, off - math.inf)
            some = on.any(1)
            for h in range(Hq):
                q = st["q"][b, h, i0:i1].double()
                k, v = (st[n][b, h // G, j0:j1].double() for n in ("k", "v"))
                s = torch.einsum("id,jd->ij", q, k) / (8.0 * case["eps"]) + bias
                z = torch.where(some, torch.logsumexp(s, 1), off)
                w = torch.exp(s - z[:, None])
                o = w @ v
                out["o"][b, h, i0:i1], out["u"][b, h, i0:i1] = o, -z
                if step:
                    g = st["dO"][b, h, i0:i1].double()
                    e = w * (g @ v.T - (g * o).sum(1, keepdim=True)) / (8.0 * case["eps"])
                    out["dq"][b, h, i0:i1] = e @ k
                    out["dk"][b, h // G, j0:j1] += e.T @ q
                    out["dv"][b, h // G, j0:j1] += w.T @ g
    return out
