"""Softmax attention and rotary positions on a GPU against the float64 forms,
within bounds that count roundings (tests/softmax_ref.py)."""
import math

import pytest
import torch

from tests import softmax_ref as ref

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
TYPES = [pytest.param(F32, id="f32"), pytest.param(BF16, id="bf16")]


def draw(dtype, B, Hq, Hk, Lq, Lk, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda h, n: torch.randn(B, h, n, 64, generator=g, device="cuda").to(dtype)
    return r(Hq, Lq), r(Hk, Lk), r(Hk, Lk), r(Hq, Lq)


def check(q, k, v, dO, *, backward=True, eps=1.0, **kw):
    """Forward (and backward) of the library against float64; returns the results."""
    import banded_log_domain_b200 as sa

    dt = q.dtype
    o, u = sa.sinkhorn_attn_softmax_fwd(q, k, v, eps=eps, **kw)
    wo, wu, P = ref.forward(q, k, v, eps=eps, **kw)
    lim = ref.bounds(q, k, v, dO if backward else None, P, dt, eps=eps)
    ref.close("o", o, wo, lim["o"], dt)
    assert float((u.double() - wu).abs().max()) <= ref.U_ATOL
    none = ~ref.support(q.shape[0], q.shape[2], k.shape[2], kw["W"], kw.get("causal", False),
                        kw.get("mask"), kw.get("q_pos"), q.device).any(-1)
    none = none[:, None].expand(u.shape)
    assert bool((u[none] == 0).all()) and bool((o[none] == 0).all())
    if not backward:
        return o, u
    dq, dk, dv = sa.sinkhorn_attn_softmax_bwd(q, k, v, o, dO, u, eps=eps, **kw)
    want = ref.backward(q, k, v, dO, P, eps=eps)
    for n, x, w in zip(("dq", "dk", "dv"), (dq, dk, dv), want):
        ref.close(n, x, w, lim[n], dt)
    assert bool((dq[none] == 0).all())
    return o, u, dq, dk, dv


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("L,W", [(1, 0), (1, 9), (2, 1), (7, 0), (63, 5), (64, 64), (65, 3), (127, 31),
                                 (129, 128), (257, 40), (300, 1000), (513, 100), (700, 255)])
def test_lengths_and_bands(dtype, L, W, causal):
    check(*draw(dtype, 2, 2, 2, L, L, seed=L + W), W=W, causal=causal)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (2, 1), (3, 1), (6, 2), (5, 1), (8, 1), (40, 2), (64, 1), (33, 1)])
def test_shared_key_heads(dtype, Hq, Hk):
    check(*draw(dtype, 2, Hq, Hk, 75, 75, seed=Hq), W=20, causal=False)
    check(*draw(dtype, 1, Hq, Hk, 150, 150, seed=Hq), W=150, causal=True)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("kind", ["tail", "holes", "one", "none", "head"])
@pytest.mark.parametrize("W", [3, 300])
def test_masks(dtype, kind, W):
    B, L = 3, 300
    x = draw(dtype, B, 4, 2, L, L, seed=5)
    j = torch.arange(L, device="cuda")[None]
    n = torch.tensor([[300], [200], [1]], device="cuda")
    mask = {"tail": j < n, "head": j >= 300 - n, "one": j == n - 1, "none": j < 0 * n,
            "holes": torch.rand(B, L, generator=torch.Generator("cuda").manual_seed(1),
                                device="cuda") < 0.3}[kind].to(torch.uint8)
    # what masked tokens hold is not used: infinities and NaN
    bad = torch.tensor([float("nan"), float("inf"), -float("inf")], device="cuda").to(dtype)
    q, k, v, dO = (t.clone() for t in x)
    fill = bad[torch.arange(64, device="cuda") % 3]
    for t in (q, k, v, dO):
        t.copy_(torch.where(mask[:, None, :, None] != 0, t, fill))
    got = check(q, k, v, dO, W=W, mask=mask)
    off = mask == 0
    for t in got[2:]:  # masked tokens' gradients
        assert bool((t[off[:, None].expand(t.shape[:3])] == 0).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("L", [60, 130])
@pytest.mark.parametrize("W", [3, 130])
def test_masks_of_small_problems(dtype, L, W):
    # fp32 tiles of 16 and of 32 rows
    q, k, v, dO = draw(dtype, 3, 4, 2, L, L, seed=L)
    mask = (torch.rand(3, L, generator=torch.Generator("cuda").manual_seed(W), device="cuda") < 0.5).to(torch.uint8)
    mask[2] = 0
    off = (mask == 0)[:, None, :, None]
    for i, t in enumerate((q, k, v, dO)):
        t.masked_fill_(off, (float("nan"), float("inf"))[i % 2])
    for causal in (False, True):
        check(q, k, v, dO, W=W, mask=mask, causal=causal)


@pytest.mark.parametrize("W", [30, 300])
def test_gradients_of_peaked_rows(W):
    # A rounding to bf16 is off by e = 1.66e-3 of a value in the root mean square; dS is
    # rounded in front of a product with normal numbers, the result once more: sqrt(2) e =
    # 2.35e-3 of the gradient's norm, a tenth more allowed.  (D from the rounded O alone,
    # wrong by e |D| in every entry of a row, would make it 2.9e-3 at this temperature.)
    import banded_log_domain_b200 as sa

    q, k, v, dO = draw(BF16, 2, 4, 4, 300, 300, seed=21)
    kw = dict(W=W, eps=0.5, causal=True)
    o, u = sa.sinkhorn_attn_softmax_fwd(q, k, v, **kw)
    got = sa.sinkhorn_attn_softmax_bwd(q, k, v, o, dO, u, **kw)
    want = ref.backward(q, k, v, dO, ref.forward(q, k, v, **kw)[2], eps=0.5)
    for name, x, w in zip(("dq", "dk"), got, want):
        assert float((x.double() - w).norm() / w.norm()) < 2.6e-3, name


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("eps", [2.0 ** -20, 2.0 ** 30, 2.0 ** 100])
def test_temperatures_far_from_one(dtype, eps):
    # q grows with eps, so that the scores stay; at 2^100 it cannot, and they vanish
    q, k, v, dO = draw(dtype, 1, 2, 2, 150, 150, seed=3)
    f = eps if eps < 2.0 ** 40 else 1.0
    check(q * f, k, v, dO, W=70, eps=eps)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("log2_eps", [-10, -20, -24, -28, -30, -33, -40, -60, -100])
@pytest.mark.parametrize("Hq,Lq,Lk,W", [(2, 200, 200, 200), (2, 300, 300, 40), (4, 40, 3000, 3000), (2, 1, 3000, 3000),
                                        (16, 2500, 2500, 60)])
def test_scores_of_any_size(dtype, log2_eps, Hq, Lq, Lk, W):
    # Small whole numbers and a power of two for c: <q, k> is exact and differs by 1
    # at least, S by 2^10 / 8, so P is 1 / (keys that share the maximum) and 0
    # elsewhere, for scores of up to 2^9 2^97.  O errs as bounds() says, with s = 0 in
    # it.  u = -(max S + ln ties): its constants, products and sum round six times.
    import banded_log_domain_b200 as sa

    g = torch.Generator(device="cuda").manual_seed(Lk)
    r = lambda h, n: torch.randint(-3, 4, (1, h, n, 64), generator=g, device="cuda").to(dtype)
    q, k = r(Hq, Lq), r(2, Lk)
    v = torch.randn(1, 2, Lk, 64, generator=g, device="cuda").to(dtype)
    eps = 2.0 ** log2_eps
    o, u = sa.sinkhorn_attn_softmax_fwd(q, k, v, W=W, eps=eps, causal=True)
    kk, vv = (t.double().repeat_interleave(Hq // 2, 1) for t in (k, v))
    S = q.double() @ kk.transpose(-1, -2)
    S.masked_fill_(~ref.support(1, Lq, Lk, W, True, None, None, "cuda")[:, None], -float("inf"))
    top = S.amax(-1, keepdim=True)
    ties = (S == top).double()
    P = ties / ties.sum(-1, keepdim=True)
    ref.close("o", o, P @ vv, (ref.H[dtype] + ref.S) * (P @ vv.abs()), dtype)
    want = -(top[..., 0] / (8 * eps) + torch.log(ties.sum(-1)))
    assert bool(torch.isfinite(u).all())
    assert bool(((u.double() - want).abs() <= 6 * 2.0 ** -24 * want.abs() + ref.U_ATOL).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("eps", [2.0 ** -4, 2.0 ** -7])
def test_gradients_at_large_duals(dtype, eps, monkeypatch):
    # P = exp(S + u) from an fp32 u: u passes seven roundings on its way from the maximum to
    # the exponent (c2, the product, the sum, ln 2 and its product, 1 / c, c2 again), 2^-21 |u|
    # in all; the score's own, of 64 terms of random sign, 8 2^-24 sum |q k| c, is under
    # 2^-21 of |u| plus that sum / 8.  Twice that for P in the forward and here.
    import banded_log_domain_b200 as sa

    q, k, v, dO = draw(dtype, 1, 4, 2, 260, 260, seed=31)
    kw = dict(W=90, causal=True)
    o, u = sa.sinkhorn_attn_softmax_fwd(q, k, v, eps=eps, **kw)
    wo, wu, P = ref.forward(q, k, v, eps=eps, **kw)
    terms = (q.double().abs() @ k.double().abs().repeat_interleave(2, 1).transpose(-1, -2)).max() / (8 * eps)
    s = float(wu.abs().max() + terms / 8) * 2.0 ** -21
    assert float((u.double() - wu).abs().max()) <= s
    monkeypatch.setattr(ref, "S", 2 * s)
    lim = ref.bounds(q, k, v, dO, P, dtype, eps=eps)
    ref.close("o", o, wo, lim["o"], dtype)
    got = sa.sinkhorn_attn_softmax_bwd(q, k, v, o, dO, u, eps=eps, **kw)
    for n, x, w in zip(("dq", "dk", "dv"), got, ref.backward(q, k, v, dO, P, eps=eps)):
        ref.close(n, x, w, lim[n], dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("G", [1, 4, 7])
@pytest.mark.parametrize("Lq,Lk,W", [(1, 1, 0), (1, 70, 70), (1, 1000, 1000), (1, 5000, 5000), (1, 5000, 300),
                                     (2, 130, 130), (5, 4096, 4096), (17, 3001, 3001), (40, 3001, 900)])
def test_few_queries_over_a_cache(dtype, G, Lq, Lk, W):
    # ragged caches; what lies behind a sequence's last token is not used
    B = 3
    q, k, v, dO = draw(dtype, B, 2 * G, 2, Lq, Lk, seed=Lk)
    q_pos = torch.tensor([Lk - Lq, (Lk - Lq) // 2, 0], dtype=torch.int32, device="cuda")
    behind = torch.arange(Lk, device="cuda")[None] >= q_pos[:, None] + Lq
    for t in (k, v):
        t.masked_fill_(behind[:, None, :, None], float("nan"))
    check(q, k, v, dO, W=W, causal=True, q_pos=q_pos)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("causal", [False, True])
def test_positions_outside_the_keys(dtype, causal):
    x = draw(dtype, 6, 2, 1, 20, 150, seed=2)
    big = 2 ** 31 - 1
    q_pos = torch.tensor([-10, 140, 150, -20, big, -big - 1], dtype=torch.int32, device="cuda")
    check(*x, W=30, causal=causal, q_pos=q_pos)
    check(*x, W=2 ** 31 - 1, causal=causal, q_pos=q_pos)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("eps", [0.25, 4.0])
def test_temperature_and_large_scores(dtype, eps):
    q, k, v, dO = draw(dtype, 1, 2, 2, 200, 200, seed=9)
    check(q, k, v, dO, W=200, eps=eps)
    # scores far from zero, still summing: every row's maximum is elsewhere in the row
    check(q * 0 + 1, k + 30, v, dO, W=200, eps=100.0)


@pytest.mark.parametrize("dtype", TYPES)
def test_strided_tensors(dtype):
    import banded_log_domain_b200 as sa

    B, Hq, Hk, L = 2, 6, 2, 133
    q, k, v, dO = draw(dtype, B, Hq, Hk, L, L, seed=4)
    kw = dict(W=50, causal=True)
    want = check(q, k, v, dO, **kw)

    def blhd(t):  # the same values as a slice of a [B, L, H + 1, 2 d] buffer
        x = torch.full((t.shape[0], t.shape[2], t.shape[1] + 1, 128), float("nan"), dtype=dtype, device="cuda")
        y = x[:, :, 1:, 64:].transpose(1, 2)
        y.copy_(t)
        return y, x

    (sq, _), (sk, _), (sv, _), (sg, _) = (blhd(t) for t in (q, k, v, dO))
    (so, ob), (sdq, qb), (sdk, kb), (sdv, vb) = (blhd(torch.zeros_like(t)) for t in (q, q, k, k))
    o, u = sa.sinkhorn_attn_softmax_fwd(sq, sk, sv, o=so, **kw)
    got = sa.sinkhorn_attn_softmax_bwd(sq, sk, sv, o, sg, u, dq=sdq, dk=sdk, dv=sdv, **kw)
    assert o is so and got[0] is sdq
    for a, b in zip((o, u) + got, want):
        assert torch.equal(a, b)
    for buf in (ob, qb, kb, vb):  # nothing beside the views was written
        assert bool(torch.isnan(buf[:, :, 0]).all()) and bool(torch.isnan(buf[..., :64]).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_offsets_beyond_32_bits(dtype):
    # a cache whose tokens lie 2^17 elements apart: the last ones are past 2^31 elements
    import banded_log_domain_b200 as sa

    L = 17000
    q, k, v, dO = draw(dtype, 1, 2, 1, 200, L, seed=11)
    big = torch.empty(L << 17, dtype=dtype, device="cuda")
    kb = big.as_strided((1, 1, L, 64), (L << 17, L << 17, 1 << 17, 1))
    vb = big.as_strided((1, 1, L, 64), (L << 17, L << 17, 1 << 17, 1), 64)
    kb.copy_(k)
    vb.copy_(v)
    for n in (1, 200):  # single tokens, and tiles
        kw = dict(W=300, causal=True)
        o, u = sa.sinkhorn_attn_softmax_fwd(q[:, :, 200 - n:], kb, vb, **kw)
        wo, wu = sa.sinkhorn_attn_softmax_fwd(q[:, :, 200 - n:], k, v, **kw)
        assert torch.equal(o, wo) and torch.equal(u, wu)
    g = sa.sinkhorn_attn_softmax_bwd(q, kb, vb, o, dO, u, **kw)
    assert all(torch.equal(x, y) for x, y in zip(g, sa.sinkhorn_attn_softmax_bwd(q, k, v, o, dO, u, **kw)))
    freqs, _ = sa.sinkhorn_attn_rotary_freqs(64)
    r, _ = sa.sinkhorn_attn_rotary_fwd(kb, None, freqs)
    assert torch.equal(r, sa.sinkhorn_attn_rotary_fwd(k, None, freqs)[0])
    sa.sinkhorn_attn_rotary_fwd(kb, None, freqs, q_out=vb)
    assert torch.equal(vb, r)


@pytest.mark.parametrize("dtype", TYPES)
def test_a_longer_problem_and_a_head_of_it(dtype):
    # The bounds of the whole and of one key head with its two query heads alone.  The
    # two need not be equal to the bit: how many row tiles share an item, and with
    # it the order in which a row's chunks are joined, goes by the number of tiles.
    q, k, v, dO = draw(dtype, 1, 4, 2, 5000, 5000, seed=6)
    check(q, k, v, dO, W=200)
    check(q[:, 2:], k[:, 1:], v[:, 1:], dO[:, 2:], W=200)


@pytest.mark.parametrize("dtype", TYPES)
def test_a_nan_in_use_is_seen_and_stays_with_its_sequence(dtype):
    import banded_log_domain_b200 as sa

    q, k, v, dO = draw(dtype, 2, 2, 2, 600, 600, seed=8)
    v[0, 0, 300, 3] = float("nan")
    k[1, 1, 10, 0] = float("nan")
    o, u = sa.sinkhorn_attn_softmax_fwd(q, k, v, W=20)
    assert bool(torch.isnan(o[0, 0, 280:321, 3]).all())
    assert bool(torch.isnan(o[1, 1, :31]).all()) and bool(torch.isnan(u[1, 1, :31]).all())
    assert bool(torch.isfinite(o[0, 1]).all()) and bool(torch.isfinite(o[1, 0]).all())
    # at most 255 positions past the band
    assert bool(torch.isfinite(o[0, 0, :280 - 255]).all()) and bool(torch.isfinite(o[0, 0, 321 + 255:]).all())
    assert bool(torch.isfinite(o[1, 1, 31 + 255:]).all()) and bool(torch.isfinite(u[0]).all())


@pytest.mark.parametrize("dtype", TYPES)
def test_same_results_again_in_a_graph_and_on_two_streams(dtype):
    import banded_log_domain_b200 as sa

    probs = [draw(dtype, 2, 4, 2, 400, 400, seed=s) for s in (1, 2)] + \
        [draw(dtype, 2, 4, 2, 1, 6000, seed=3)]
    kws = [dict(W=100), dict(W=400, causal=True), dict(W=6000, causal=True)]

    def step(x, kw):
        q, k, v, dO = x
        o, u = sa.sinkhorn_attn_softmax_fwd(q, k, v, **kw)
        return (o, u) + sa.sinkhorn_attn_softmax_bwd(q, k, v, o, dO, u, **kw)

    want = [step(*z) for z in zip(probs, kws)]
    streams = [torch.cuda.Stream() for _ in probs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(3):
        for s, x, kw in zip(streams, probs, kws):
            with torch.cuda.stream(s):
                got.append(step(x, kw))
    torch.cuda.synchronize()
    for n, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[n % 3]))
    for x, kw, w in zip(probs, kws, want):
        graph = torch.cuda.CUDAGraph()
        live = [t.clone() for t in x]
        with torch.cuda.graph(graph):
            out = step(live, kw)
        for t in live:
            t.neg_()
        graph.replay()
        for t, y in zip(live, x):
            t.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, w))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Lq,Lk,H", [(4, 40000, 1), (16, 20000, 1), (70, 9000, 2), (300, 3000, 1), (1100, 1100, 1)])
def test_split_keys_of_few_rows(dtype, Lq, Lk, H):
    # the parts of a row's keys, forward and (fp32) backward; where most tokens are
    # masked there are fewer chunks than blocks
    q, k, v, dO = draw(dtype, 1, H, H, Lq, Lk, seed=Lq)
    check(q, k, v, dO, W=Lk)
    mask = torch.ones(1, Lk, dtype=torch.uint8, device="cuda")
    mask[:, :Lk - Lq - 100] = 0
    for _ in range(3):  # workspaces that held other parts
        check(q, k, v, dO, W=Lk, mask=mask, causal=True)
        check(q, k, v, dO, W=Lk, mask=mask)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Hq,Hk,Lq,Lk,W,masked", [(2, 1, 1, 5000, 5000, False), (2, 1, 2, 5000, 5000, True),
                                                  (8, 1, 3, 700, 30, True), (4, 1, 40, 3000, 3000, False),
                                                  (2, 2, 300, 900, 900, True), (2, 2, 500, 500, 20, False)])
def test_a_workspace_may_hold_anything(dtype, Hq, Hk, Lq, Lk, W, masked):
    import banded_log_domain_b200 as sa

    q, k, v, dO = draw(dtype, 2, Hq, Hk, Lq, Lk, seed=Lq)
    mask = (torch.rand(2, Lk, generator=torch.Generator("cuda").manual_seed(2), device="cuda") < 0.05).to(torch.uint8)
    kw = dict(W=W, mask=mask if masked else None, q_pos=torch.tensor([Lk - Lq, Lk // 7], dtype=torch.int32, device="cuda"))
    p = sa._softmax_params(q, k, v, W, 1.0, False)
    f, b = sa.sinkhorn_attn_softmax_workspace_size(p)
    got = []
    for fill in (0, 0xff):  # zeros, and NaN
        ws = torch.full((max(f, b),), fill, dtype=torch.uint8, device="cuda")
        o, u = sa.sinkhorn_attn_softmax_fwd(q, k, v, ws=ws, **kw)
        ws.fill_(fill)
        got.append((o, u) + sa.sinkhorn_attn_softmax_bwd(q, k, v, o, dO, u, ws=ws, **kw))
    assert all(torch.equal(x, y) for x, y in zip(*got))
    assert all(bool(torch.isfinite(x).all()) for x in got[0])


def test_workspace_status_and_reuse():
    import banded_log_domain_b200 as sa

    q, k, v, dO = draw(BF16, 1, 2, 2, 1, 9000, seed=3)
    p = sa._softmax_params(q, k, v, 9000, 1.0, True)
    f, b = sa.sinkhorn_attn_softmax_workspace_size(p)
    ws = torch.full((max(f, b),), 0x5a, dtype=torch.uint8, device="cuda")  # needs no initialisation
    kw = dict(W=9000, causal=True)
    o, u = sa.sinkhorn_attn_softmax_fwd(q, k, v, ws=ws, **kw)
    assert sa.sinkhorn_attn_poll(ws) == 0
    w = sa.sinkhorn_attn_softmax_fwd(q, k, v, **kw)
    assert torch.equal(o, w[0]) and torch.equal(u, w[1])
    g = sa.sinkhorn_attn_softmax_bwd(q, k, v, o, dO, u, ws=ws, **kw)
    assert sa.sinkhorn_attn_poll(ws) == 0
    assert all(torch.equal(a, c) for a, c in zip(g, sa.sinkhorn_attn_softmax_bwd(q, k, v, o, dO, u, **kw)))
    with pytest.raises(sa.SinkhornAttnError) as e:
        sa.sinkhorn_attn_softmax_fwd(q, k, v, ws=ws[:f - 1], **kw)
    assert e.value.status == -3


@pytest.mark.parametrize("B,H,Lq,Lk", [(1, 2, 0, 0), (1, 2, 0, 5), (0, 2, 3, 3), (2, 0, 3, 5)])
def test_empty_calls_reset_the_status_word(B, H, Lq, Lk):
    import banded_log_domain_b200 as sa

    q, k, v, dO = draw(BF16, B, H, H, Lq, Lk)
    u = torch.empty(B, H, Lq, device="cuda")
    for f in (lambda ws: sa.sinkhorn_attn_softmax_fwd(q, k, v, W=1, ws=ws),
              lambda ws: sa.sinkhorn_attn_softmax_bwd(q, k, v, q, dO, u, W=1, ws=ws)):
        ws = torch.full((1024,), 0x5a, dtype=torch.uint8, device="cuda")
        f(ws)
        assert sa.sinkhorn_attn_poll(ws) == 0
        f(None)


@pytest.mark.parametrize("W", [-1, -2 ** 31, -2 ** 31 - 1, -2 ** 32, -2 ** 40])
def test_negative_bands_are_refused(W):
    import banded_log_domain_b200 as sa

    q, k, v, _ = draw(F32, 1, 1, 1, 8, 8)
    with pytest.raises(sa.SinkhornAttnError) as e:
        sa.sinkhorn_attn_softmax_fwd(q, k, v, W=W)
    assert e.value.status == -1


def test_bands_past_32_bits_are_dense():
    import banded_log_domain_b200 as sa

    q, k, v, _ = draw(F32, 1, 1, 1, 8, 8)
    a, b = (sa.sinkhorn_attn_softmax_fwd(q, k, v, W=W) for W in (8, 2 ** 40))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_refusals_on_the_gpu():
    import banded_log_domain_b200 as sa

    q, k, v, dO = draw(BF16, 1, 4, 2, 8, 8)
    ok = dict(W=4)
    for bad in (dict(k=k.float()), dict(v=v[:, :, :7]), dict(q=q[..., :32]), dict(q=q.half()), dict(v=v.cpu()),
                dict(k=k[:, :1].expand(1, 2, 8, 64)), dict(q=q.transpose(2, 3).contiguous().transpose(2, 3))):
        a = dict(q=q, k=k, v=v) | bad
        with pytest.raises((ValueError, sa.SinkhornAttnError)):
            sa.sinkhorn_attn_softmax_fwd(a["q"], a["k"], a["v"], **ok)
    for kw in (dict(mask=torch.ones(1, 7, dtype=torch.uint8, device="cuda")), dict(mask=torch.ones(1, 8, device="cuda")),
               dict(mask=torch.ones(1, 8, dtype=torch.uint8)), dict(q_pos=torch.zeros(1, device="cuda")),
               dict(q_pos=torch.zeros(2, dtype=torch.int32, device="cuda")), dict(o=torch.empty_like(k)),
               dict(u=torch.empty(1, 4, 8, dtype=BF16, device="cuda"))):
        with pytest.raises(ValueError):
            sa.sinkhorn_attn_softmax_fwd(q, k, v, **ok, **kw)
    odd = torch.zeros(1, 4, 8, 65, dtype=BF16, device="cuda")
    for x in (odd[..., 1:], odd[..., :64]):  # misaligned, and strides off 16 bytes
        with pytest.raises(sa.SinkhornAttnError) as e:
            sa.sinkhorn_attn_softmax_fwd(x, k, v, **ok)
        assert e.value.status == -1
    pinned = torch.zeros(1, 2, 8, 64, dtype=BF16).pin_memory()
    with pytest.raises(ValueError):
        sa.sinkhorn_attn_softmax_fwd(q, pinned, v, **ok)
    with pytest.raises(ValueError):
        sa.sinkhorn_attn_rotary_fwd(q, k, torch.zeros(32, device="cuda"))
    with pytest.raises(sa.SinkhornAttnError):
        sa.sinkhorn_attn_rotary_fwd(q, k, torch.zeros(33, dtype=torch.float64, device="cuda"))
    with pytest.raises(ValueError):
        sa.sinkhorn_attn_rotary_fwd(q, k, torch.zeros(32, dtype=torch.float64, device="cuda"),
                                    pos=torch.zeros(1, 7, dtype=torch.int32, device="cuda"))


# ------------------------------------------------------------------ rotary positions
# |y - want| <= h |want| + 2^-20 (|x_a| + |x_b|) scale: the cosines and sines err by
# 2^-22 (the angle's float remainder 2^-25 turns, sincospif 2 ulp), two products and a sum
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 32), (64, 2), (64, 10), (64, 62), (128, 96), (8, 8), (256, 250),
                                   (72, 64), (40, 16)])
def test_rotary(dtype, interleaved, d, rot):
    import banded_log_domain_b200 as sa

    g = torch.Generator(device="cuda").manual_seed(rot)
    B, Hq, Hk, L = 2, 5, 2, 37
    q, k = (torch.randn(B, h, L, d, generator=g, device="cuda").to(dtype) for h in (Hq, Hk))
    freqs, scale = sa.sinkhorn_attn_rotary_freqs(rot, scaling="by_parts", factor=4.0, train_len=512)
    near = torch.arange(L, dtype=torch.int32, device="cuda").expand(B, L).contiguous()
    far = torch.randint(0, 2 ** 31 - 1, (B, L), generator=g, device="cuda", dtype=torch.int32)
    for pos in (None, far, -far, near):
        for f, inv in ((sa.sinkhorn_attn_rotary_fwd, False), (sa.sinkhorn_attn_rotary_bwd, True)):
            got = f(q, k, freqs, pos=pos, interleaved=interleaved, scale=scale)
            for x, y in zip((q, k), got):
                want = ref.rotate(x, freqs, near if pos is None else pos, interleaved, scale, inv)
                pair = ref.rotate(x.abs(), freqs * 0, near, interleaved, scale, inv)
                other = x.double().abs().clone()
                n = rot // 2
                i, j = (slice(0, rot, 2), slice(1, rot, 2)) if interleaved else (slice(0, n), slice(n, rot))
                other[..., i], other[..., j] = x[..., j].double().abs(), x[..., i].double().abs()
                ref.close("y", y, want, 2.0 ** -20 * (pair + scale * other), dtype)
                assert torch.equal(y[..., rot:], x[..., rot:])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rot,interleaved", [(64, False), (32, True), (6, False)])
def test_rotary_layouts_in_place_and_undone(dtype, rot, interleaved):
    import banded_log_domain_b200 as sa

    B, Hq, Hk, L = 2, 4, 1, 300
    q, k, _, _ = draw(dtype, B, Hq, Hk, L, L, seed=1)
    freqs, _ = sa.sinkhorn_attn_rotary_freqs(rot)
    kw = dict(interleaved=interleaved, scale=0.5)
    want = sa.sinkhorn_attn_rotary_fwd(q, k, freqs, **kw)
    # a [B, L, H, d] projection read in place, its results in the attention's layout
    proj = torch.cat([q, k], 1).transpose(1, 2).contiguous()
    got = sa.sinkhorn_attn_rotary_fwd(proj[:, :, :Hq].transpose(1, 2), proj[:, :, Hq:].transpose(1, 2), freqs, **kw)
    assert all(g.is_contiguous() and torch.equal(g, w) for g, w in zip(got, want))
    # queries alone; on their own storage
    alone, none = sa.sinkhorn_attn_rotary_fwd(q, None, freqs, **kw)
    assert none is None and torch.equal(alone, want[0])
    q2, k2 = q.clone(), k.clone()
    r = sa.sinkhorn_attn_rotary_fwd(q2, k2, freqs, q_out=q2, k_out=k2, **kw)
    assert r[0] is q2 and torch.equal(q2, want[0]) and torch.equal(k2, want[1])
    # the transposed rotation undoes it: two roundings of size h, and fp32 sines
    back = sa.sinkhorn_attn_rotary_bwd(*sa.sinkhorn_attn_rotary_fwd(q, k, freqs, interleaved=interleaved), freqs,
                                       interleaved=interleaved)
    h = ref.H[dtype]
    for x, y in zip((q, k), back):
        n = float(x.double().abs().max())
        assert float((x.double() - y.double()).abs().max()) <= 4 * h * n + 2.0 ** -18 * n


@pytest.mark.parametrize("inverse", [False, True])
def test_cosines_and_sines_at_far_positions(inverse):
    # Channel pairs of (1, 0) give the cosine and the sine themselves.  They err by
    # sincospif's one ulp (2^-23 at most), the half steps of the remainder's correction,
    # of the scale (1 here) and of the product with 1: 5 2^-24, and less than 2^-40 of
    # the angle.  The exact angle: whole numbers, with 2 pi to 60 digits.
    from fractions import Fraction as F

    import banded_log_domain_b200 as sa

    two_pi = 2 * F(314159265358979323846264338327950288419716939937510582097494459, 10 ** 62)
    freqs, _ = sa.sinkhorn_attn_rotary_freqs(16)
    at = [0, 1, 2, 1000, 2 ** 20 - 3, 2 ** 27 + 1, 1_000_000_007, 2 ** 31 - 1, -2 ** 31] + \
        [2 ** 31 - 1 - 12345 * i for i in range(1, 400)]
    pos = torch.tensor([at], dtype=torch.int32, device="cuda")
    q = torch.zeros(1, 1, len(at), 16, device="cuda")
    q[..., :8] = 1
    f = sa.sinkhorn_attn_rotary_bwd if inverse else sa.sinkhorn_attn_rotary_fwd
    y = f(q, None, freqs, pos=pos)[0][0, 0].double().cpu()
    want = torch.empty(len(at), 16, dtype=torch.float64)
    for t, p in enumerate(at):
        for i, w in enumerate(freqs.tolist()):
            a = F(-p if inverse else p) * F(w)
            a = float(a - two_pi * round(a / two_pi))
            want[t, i], want[t, 8 + i] = math.cos(a), math.sin(a)
    assert float((y - want).abs().max()) <= 5 * 2.0 ** -24


def test_rotary_refuses_the_pair_of_frequencies_and_factor():
    import banded_log_domain_b200 as sa

    q = torch.zeros(1, 1, 4, 64, device="cuda")
    for f in (sa.sinkhorn_attn_rotary_fwd, sa.sinkhorn_attn_rotary_bwd):
        with pytest.raises(ValueError, match="freqs"):
            f(q, q, sa.sinkhorn_attn_rotary_freqs(64))


def test_rotary_is_relative():
    # the scores of rotated queries and keys depend on the distance alone
    import banded_log_domain_b200 as sa

    q, k, _, _ = draw(F32, 1, 1, 1, 64, 64, seed=1)
    freqs, _ = sa.sinkhorn_attn_rotary_freqs(64)
    at = torch.arange(64, dtype=torch.int32, device="cuda")[None]
    s = []
    for shift in (0, 1_000_000_000):
        a, b = sa.sinkhorn_attn_rotary_fwd(q, k, freqs, pos=at + shift)
        s.append(a.double() @ b.double().transpose(-1, -2))
    # 64 products of values under 5 whose factors err by 2^-21
    assert float((s[0] - s[1]).abs().max()) <= 64 * 25 * 2.0 ** -20


@pytest.mark.parametrize("dtype", TYPES)
def test_rotary_in_a_graph_and_on_two_streams(dtype):
    import banded_log_domain_b200 as sa

    freqs, _ = sa.sinkhorn_attn_rotary_freqs(64)
    probs = [draw(dtype, 2, 4, 2, L, L, seed=L)[:2] for L in (1, 3000)]
    pos = [torch.full((2, 1), 70000, dtype=torch.int32, device="cuda"), None]

    def step(x, p):
        y = sa.sinkhorn_attn_rotary_fwd(*x, freqs, pos=p)
        return y + sa.sinkhorn_attn_rotary_bwd(*y, freqs, pos=p)

    want = [step(*z) for z in zip(probs, pos)]
    streams = [torch.cuda.Stream() for _ in probs]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(3):
        for s, x, p in zip(streams, probs, pos):
            with torch.cuda.stream(s):
                got.append(step(x, p))
    torch.cuda.synchronize()
    for n, y in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(y, want[n % 2]))
    for x, p, w in zip(probs, pos, want):
        live = [t.clone() for t in x]
        at = None if p is None else p.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step(live, at)
        for t in live:
            t.neg_()
        if at is not None:
            at.add_(5)
        graph.replay()
        for t, y in zip(live, x):
            t.copy_(y)
        if at is not None:
            at.copy_(p)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, w))


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype", TYPES)
def test_a_layer_rotary_attention_and_back(dtype):
    """Projections in [B, L, H, d] -> rotary -> attention -> gradients of the projections,
    then single tokens over the rotated keys; the Sinkhorn attention takes the same q, k."""
    import banded_log_domain_b200 as sa

    B, Hq, Hk, L = 2, 4, 2, 200
    q, k, v, dO = draw(dtype, B, Hq, Hk, L, L, seed=12)
    pq, pk, pv = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k, v))
    freqs, scale = sa.sinkhorn_attn_rotary_freqs(64, scaling="by_parts", factor=2.0, train_len=128)
    kw = dict(W=64, causal=True)
    rq, rk = sa.sinkhorn_attn_rotary_fwd(pq, pk, freqs, scale=scale)
    o, u, dq, dk, dv = check(rq, rk, pv, dO, **kw)
    gq, gk = sa.sinkhorn_attn_rotary_bwd(dq, dk, freqs, scale=scale)
    # float64 from the projections on: autograd through both
    leaves = [t.double().requires_grad_() for t in (q, k, v)]
    at = torch.arange(L, device="cuda").expand(B, L)
    a, b = (ref.rotate(t, freqs, at, False, scale, False) for t in leaves[:2])
    wo, wu, _ = ref.forward(a, b, leaves[2], **kw)
    want = torch.autograd.grad((wo * dO.double()).sum(), leaves)
    wo, wu = wo.detach(), wu.detach()
    # every tensor is rounded to the type at most six times on the way (rq, rk, P, dS, o, dq, gq)
    tol = 6 * ref.H[dtype] + 2.0 ** -14
    for x, w in zip((o, u, gq, gk, dv), (wo, wu) + tuple(want)):
        assert float((x.double() - w).norm() / w.norm()) <= tol
    # the last tokens one at a time over the cache of rotated keys
    for t in (0, 1, 64, 199):
        pos = torch.full((B, 1), t, dtype=torch.int32, device="cuda")
        q1, _ = sa.sinkhorn_attn_rotary_fwd(pq[:, :, t:t + 1], None, freqs, pos=pos, scale=scale)
        assert torch.equal(q1, rq[:, :, t:t + 1])
        o1, u1 = sa.sinkhorn_attn_softmax_fwd(q1, rk, pv, q_pos=pos[:, 0].contiguous(), **kw)
        assert float((u1 - u[:, :, t:t + 1]).abs().max()) <= 2 * ref.U_ATOL
        # both round P (at another maximum) and O
        assert float((o1.double() - o[:, :, t:t + 1].double()).norm() / wo[:, :, t:t + 1].norm()) <= tol
    if Hq != Hk:
        rk2 = rk.repeat_interleave(Hq // Hk, 1)
        v2 = v.repeat_interleave(Hq // Hk, 1)
        so, st = sa.sinkhorn_attn_fwd(rq, rk2, v2, W=64, eps=1.0, T=2, R=2)
        assert bool(torch.isfinite(so).all()) and bool(torch.isfinite(st).all())


def test_the_readme_runs():
    # its Python examples, one after the other as a reader would type them
    import os
    import re

    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    assert len(blocks) >= 2
    names = {}
    for block in blocks:
        exec(block, names)
    for n in ("o", "u", "dq", "dk", "dv"):
        assert bool(torch.isfinite(names[n]).all())
    assert names["dq"].shape == names["q"].shape and names["dk"].shape == names["k"].shape
