"""Softmax attention and rotary positions without a GPU: the float64 forms the
GPU tests compare with, argument checks, sizes and the frequencies."""
import ctypes
import math
import random

import pytest
import torch

import banded_log_domain_b200 as sa
from tests import softmax_ref as ref


def P(B=2, Hq=4, Hk=2, Lq=50, Lk=100, d=64, W=7, eps=1.0, causal=0, dtype=sa.SA_BF16):
    return sa.sa_softmax_params(B, Hq, Hk, Lq, Lk, d, W, eps, causal, dtype)


def R(B=2, Hq=4, Hk=2, L=50, d=64, rot=64, interleaved=0, scale=1.0, dtype=sa.SA_BF16):
    return sa.sa_rotary_params(B, Hq, Hk, L, d, rot, interleaved, scale, dtype)


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), -1), (dict(W=-1), -1), (dict(eps=0.0), -1), (dict(eps=float("nan")), -1),
    (dict(eps=float("inf")), -1), (dict(causal=2), -1), (dict(dtype=2), -1), (dict(Lq=101), -1),
    (dict(Hq=5), -1), (dict(Hk=0), -1), (dict(d=0), -1), (dict(d=32), -2), (dict(d=128), -2),
    (dict(Hq=130, Hk=2), -2), (dict(B=40000), -2), (dict(Lk=(1 << 30) + 1), -2),
])
def test_bad_sizes_are_refused(kw, status):
    lib = sa.load()
    p = P(**kw)
    assert lib.sinkhorn_attn_softmax_workspace_size(ctypes.byref(p), None, None) == status
    assert lib.sinkhorn_attn_softmax_fwd(ctypes.byref(p), *[None] * 8, 1 << 40, None) == status
    assert lib.sinkhorn_attn_softmax_bwd(ctypes.byref(p), *[None] * 12, 1 << 40, None) == status


@pytest.mark.parametrize("eps,status", [(2.0 ** -100, 0), (2.0 ** 100, 0), (2.0 ** -101, -2), (2.0 ** 101, -2),
                                        (1e-45, -2), (3.4e38, -2)])
def test_temperatures_at_the_ends_of_fp32_are_refused(eps, status):
    lib = sa.load()
    for dt in (sa.SA_F32, sa.SA_BF16):
        assert lib.sinkhorn_attn_softmax_workspace_size(ctypes.byref(P(eps=eps, dtype=dt)), None, None) == status


def test_null_params_small_workspace_and_host_pointers():
    lib = sa.load()
    assert lib.sinkhorn_attn_softmax_fwd(None, *[None] * 8, 1 << 40, None) == -1
    assert lib.sinkhorn_attn_softmax_bwd(None, *[None] * 12, 1 << 40, None) == -1
    p = P()
    f, b = sa.sinkhorn_attn_softmax_workspace_size(p)
    assert b == 512 + 2 * 4 * 50 * 32  # status, spans, 32 bytes per query row
    assert sa.sinkhorn_attn_softmax_workspace_size(P(dtype=sa.SA_F32))[1] == 512 + (2 * 4 * 50 * 4 + 255) // 256 * 256
    assert lib.sinkhorn_attn_softmax_fwd(ctypes.byref(p), *[None] * 8, f - 1, None) == -3
    assert lib.sinkhorn_attn_softmax_bwd(ctypes.byref(p), *[None] * 12, b - 1, None) == -3
    assert lib.sinkhorn_attn_softmax_fwd(ctypes.byref(p), *[None] * 8, f, None) == -1
    assert lib.sinkhorn_attn_softmax_bwd(ctypes.byref(p), *[None] * 12, b, None) == -1
    buf = torch.zeros(2 * 4 * 100 * 64 * 4)
    a = buf.data_ptr()
    assert lib.sinkhorn_attn_softmax_fwd(ctypes.byref(p), a, a, a, None, None, a, a, a, f, None) == -1
    assert lib.sinkhorn_attn_softmax_bwd(ctypes.byref(p), a, a, a, None, None, *[a] * 7, b, None) == -1


def test_empty_problems_succeed():
    lib = sa.load()
    for kw in (dict(B=0), dict(Lq=0, Lk=0), dict(Hq=0, Hk=0)):
        p = P(**kw)
        f, b = sa.sinkhorn_attn_softmax_workspace_size(p)
        assert lib.sinkhorn_attn_softmax_fwd(ctypes.byref(p), *[None] * 8, f, None) == 0
        assert lib.sinkhorn_attn_softmax_bwd(ctypes.byref(p), *[None] * 12, b, None) == 0
    assert lib.sinkhorn_attn_softmax_fwd(ctypes.byref(P(Lq=0)), *[None] * 8, 512, None) == 0


@pytest.mark.parametrize("stride", [(-6400, 640, 64), (6400, 0, 64), (6400, 640, 60), (1 << 39, 640, 64)])
@pytest.mark.parametrize("which", ["q", "k", "v", "o", "dO", "dq", "dk", "dv"])
def test_bad_strides_are_refused(which, stride):
    lib = sa.load()
    p = P()
    setattr(p, which + "_stride", sa._S3(*stride))
    if which in "qkvo":
        assert lib.sinkhorn_attn_softmax_fwd(ctypes.byref(p), *[None] * 8, 1 << 40, None) == -1
    assert lib.sinkhorn_attn_softmax_bwd(ctypes.byref(p), *[None] * 12, 1 << 40, None) == -1


def test_workspace_is_bounded_and_grows_with_the_rows_only():
    # single tokens: parts of the rows, within the stated bound whatever the cache
    for Lk in (128, 4096, 1 << 20, 1 << 26):
        for B in (1, 3, 64, 147):
            f, _ = sa.sinkhorn_attn_softmax_workspace_size(P(B=B, Hq=64, Hk=1, Lq=1, Lk=Lk, W=Lk))
            assert f <= 37 << 20
    for dt in (sa.SA_F32, sa.SA_BF16):
        for Lq in (1, 8, 100, 1000, 4000):
            for H in (1, 8, 100):
                q = P(B=1, Hq=H, Hk=H, Lq=Lq, Lk=1 << 20, W=1 << 20, dtype=dt)
                f, b = sa.sinkhorn_attn_softmax_workspace_size(q)
                rows = 512 + (H * Lq * (32 if dt == sa.SA_BF16 else 4) + 255) // 256 * 256
                assert f <= 37 << 20 and rows <= b <= rows + (10 << 20)
    f, b = sa.sinkhorn_attn_softmax_workspace_size(P(B=1, Hq=16, Hk=16, Lq=32768, Lk=32768, W=256))
    assert f == 512 and b == 512 + 16 * 32768 * 32


def test_the_parts_stay_within_what_the_header_says():
    # 148 SMs.  Forward: a part of a row is 64 floats and two more, 264 bytes.  Tiled: two
    # blocks an SM, of 256 rows at most (items of four row tiles are never split);
    # single tokens: 296 blocks and up to 4096 key heads, 16 rows.  Backward, fp32:
    # 296 parts of 64 query rows (256 bytes) or 64 key rows (512 bytes).
    fwd = max(296 * 256, (296 + 4096) * 16) * 264
    bwd = 296 * 64 * 512
    assert fwd <= 20.1e6 and bwd <= 9.8e6
    rng = random.Random(4)
    log = lambda a, b: int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))
    for _ in range(20000):
        dt = rng.choice([sa.SA_F32, sa.SA_BF16])
        G, B, Hk = (rng.choice(x) for x in ([1, 2, 3, 4, 7, 8, 16, 33, 64], [1, 2, 8, 64, 147], [1, 2, 8, 37, 64]))
        if B * G * Hk > 65535:
            continue
        Lk = log(1, 1 << 30)
        Lq = min(Lk, log(1, 1 << 16))
        kw = dict(B=B, Hq=G * Hk, Hk=Hk, Lq=Lq, Lk=Lk, W=rng.choice([Lk, log(1, Lk)]), causal=rng.randint(0, 1), dtype=dt)
        p = P(**kw)
        if sa.load().sinkhorn_attn_softmax_workspace_size(ctypes.byref(p), None, None) != 0:
            continue
        f, b = sa.sinkhorn_attn_softmax_workspace_size(p)
        own = B * G * Hk * Lq * (32 if dt == sa.SA_BF16 else 4)
        head = 256 + (B * 8 + 255) // 256 * 256
        assert f - head <= fwd + 512, kw  # both arrays of the parts end on 256 bytes
        assert b - head - own <= (0 if dt == sa.SA_BF16 else bwd) + 512, kw


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), -1), (dict(L=-1), -1), (dict(rot=0), -1), (dict(rot=63), -1), (dict(rot=66), -1),
    (dict(interleaved=2), -1), (dict(dtype=9), -1), (dict(scale=float("inf")), -1),
    (dict(d=68, rot=64), -2), (dict(d=264, rot=64), -2), (dict(B=65536), -2), (dict(Hq=65536), -2),
    (dict(L=(1 << 30) + 1), -2),
    (dict(), -1),  # null pointers
])
def test_rotary_refuses(kw, status):
    lib = sa.load()
    for f in (lib.sinkhorn_attn_rotary_fwd, lib.sinkhorn_attn_rotary_bwd):
        assert f(ctypes.byref(R(**kw)), *[None] * 7) == status
        assert f(None, *[None] * 7) == -1
    p = R()
    p.k_stride = sa._S3(6400, 640, 60)
    assert lib.sinkhorn_attn_rotary_fwd(ctypes.byref(p), *[None] * 7) == -1
    assert lib.sinkhorn_attn_rotary_fwd(ctypes.byref(R(B=0)), *[None] * 7) == 0
    assert lib.sinkhorn_attn_rotary_fwd(ctypes.byref(R(L=0)), *[None] * 7) == 0


def test_rotary_frequencies():
    f, s = sa.sinkhorn_attn_rotary_freqs(8, base=100.0, device="cpu")
    assert s == 1.0 and f.dtype == torch.float64
    assert torch.allclose(f, 100.0 ** (-torch.arange(4, dtype=torch.float64) / 4), rtol=1e-14, atol=0)
    lin, _ = sa.sinkhorn_attn_rotary_freqs(8, base=100.0, scaling="linear", factor=4.0, device="cpu")
    assert torch.allclose(lin, f / 4, rtol=1e-14, atol=0)
    # ntk: the fastest pair is kept and the slowest is divided by the factor
    ntk, _ = sa.sinkhorn_attn_rotary_freqs(8, base=100.0, scaling="ntk", factor=4.0, device="cpu")
    assert abs(ntk[0] - f[0]) < 1e-14 and abs(ntk[3] / (f[3] / 4) - 1) < 1e-13
    # by parts: pairs that turn often are kept, slow ones are divided
    bp, s = sa.sinkhorn_attn_rotary_freqs(64, scaling="by_parts", factor=8.0, train_len=4096,
                                          device="cpu")
    f, _ = sa.sinkhorn_attn_rotary_freqs(64, device="cpu")
    turns = f * 4096 / (2 * math.pi)
    assert torch.allclose(bp[turns > 45], f[turns > 45], rtol=1e-14, atol=0)
    assert torch.allclose(bp[turns < 0.7], f[turns < 0.7] / 8, rtol=1e-14, atol=0)
    assert bool((bp <= f * (1 + 1e-14)).all()) and bool((bp >= f / 8 * (1 - 1e-14)).all())
    assert abs(s - (0.1 * math.log(8.0) + 1)) < 1e-7
    one, _ = sa.sinkhorn_attn_rotary_freqs(2, scaling="ntk", factor=4.0, device="cpu")
    assert one.tolist() == [1.0]


# train_len from far too short for any turn to long enough that even the slowest pair
# turns more than turns_lo times (65536, 131072) or turns_hi times (2^22)
@pytest.mark.parametrize("rot", [2, 6, 64])
@pytest.mark.parametrize("train_len", [3, 6, 7, 100, 512, 4096, 65536, 131072, 1 << 22])
@pytest.mark.parametrize("turns", [(32.0, 1.0), (8.0, 2.0)])
def test_frequencies_by_parts_over_all_trained_lengths(rot, train_len, turns):
    factor, n = 8.0, rot // 2
    got, _ = sa.sinkhorn_attn_rotary_freqs(rot, scaling="by_parts", factor=factor, train_len=train_len,
                                           turns=turns, device="cpu")
    f, _ = sa.sinkhorn_attn_rotary_freqs(rot, device="cpu")
    # the pair index at which train_len tokens make t whole turns: base^(-i/n) train_len = 2 pi t
    at = [n * math.log(train_len / (2 * math.pi * t), 10000.0) for t in turns]
    start, end = max(0, math.floor(at[0])), min(rot - 1, math.ceil(at[1]))
    for i in range(n):
        count = float(f[i]) * train_len / (2 * math.pi)
        share = float(got[i] / f[i])
        if count > turns[0]:
            assert abs(share - 1) < 1e-13
        elif count < turns[1]:
            assert abs(share * factor - 1) < 1e-13
        else:
            ramp = (i - start) / (end - start)
            assert 0 <= ramp <= 1 and abs(share - (ramp / factor + 1 - ramp)) < 1e-13


@pytest.mark.parametrize("kw", [
    dict(rot=0), dict(rot=7), dict(rot=8, base=1.0), dict(rot=8, base=float("inf")),
    dict(rot=8, factor=0.5), dict(rot=8, factor=float("nan")),
    dict(rot=8, scaling="by_parts", factor=2.0),
    dict(rot=8, scaling="by_parts", factor=2.0, train_len=64, turns=(1.0, 1.0)),
    dict(rot=8, scaling="by_parts", factor=2.0, train_len=64, turns=(1.0, 0.0)),
])
def test_rotary_frequencies_refuse(kw):
    with pytest.raises(sa.SinkhornAttnError) as e:
        sa.sinkhorn_attn_rotary_freqs(kw.pop("rot"), device="cpu", **kw)
    assert e.value.status == -1


def test_unknown_scalings_are_refused():
    for scaling in ("none", "yarn", None, 2):
        with pytest.raises(ValueError, match="by_parts"):
            sa.sinkhorn_attn_rotary_freqs(64, scaling=scaling, device="cpu")


def test_python_checks():
    q = torch.zeros(1, 2, 4, 64)
    with pytest.raises(ValueError):
        sa.sinkhorn_attn_softmax_fwd(q, q, q, W=1)  # host tensors
    with pytest.raises(ValueError):
        sa.sinkhorn_attn_rotary_fwd(q, q, torch.zeros(32, dtype=torch.float64))
    p = P()
    with pytest.raises(ValueError):  # an expanded tensor is never taken for a contiguous one
        sa._strided(p, "q", torch.zeros(1, 1, 1, 64).expand(2, 4, 50, 64))
    with pytest.raises(ValueError):
        sa._strided(p, "q", torch.zeros(2, 4, 64, 50).transpose(2, 3))


# ------------------------------------------------------------------ the float64 forms
def draw(B, Hq, Hk, Lq, Lk, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda h, n: torch.randn(B, h, n, 64, generator=g, dtype=torch.float64)
    return r(Hq, Lq), r(Hk, Lk), r(Hk, Lk), r(Hq, Lq)


def test_reference_is_the_row_half_of_a_sinkhorn_iteration(oracle_mod):
    # the first row update from v = 0 is u1 = -LSE_j(S), the softmax's row dual
    q, k, v, _ = draw(1, 2, 2, 20, 20)
    mask = (torch.arange(20) < 17).to(torch.uint8)[None]
    o, u, P = ref.forward(q, k, v, W=5, eps=0.7, mask=mask)
    _, st = oracle_mod.forward(q.float(), k.float(), v.float(), W=5, eps=0.7, T=0, R=1,
                               mask=mask)
    assert abs(torch.as_tensor(st)[:, :, 2] - u).max() < 1e-6
    assert torch.allclose(P.sum(-1), (mask[:, None] != 0).double().expand(1, 2, 20), atol=1e-12)


@pytest.mark.parametrize("causal", [False, True])
def test_reference_gradients_against_differences_and_autograd(causal):
    q, k, v, dO = draw(2, 4, 2, 5, 9, seed=3)
    mask = torch.ones(2, 9, dtype=torch.uint8)
    mask[0, 3], mask[1, 8] = 0, 0
    q_pos = torch.tensor([1, 6], dtype=torch.int32)  # the last query of sequence 1 lies outside
    kw = dict(W=2, eps=0.8, causal=causal, mask=mask, q_pos=q_pos)
    leaves = [x.clone().requires_grad_() for x in (q, k, v)]
    o, _, P = ref.forward(*leaves, **kw)
    auto = torch.autograd.grad((o * dO).sum(), leaves)
    formula = ref.backward(q, k, v, dO, P.detach(), eps=0.8)
    f = lambda *x: float((ref.forward(*x, **kw)[0] * dO).sum())
    for n, (a, b) in enumerate(zip(auto, formula)):
        assert torch.allclose(a, b, atol=1e-11)
        x = [q, k, v]
        for at in ((0, 1, 2, 5), (1, 0, 4, 60), (1, 1, 1, 0)):
            step = 1e-5
            up, down = x[n].clone(), x[n].clone()
            up[at] += step
            down[at] -= step
            d = (f(*x[:n], up, *x[n + 1:]) - f(*x[:n], down, *x[n + 1:])) / (2 * step)
            assert abs(d - float(b[at])) < 1e-8
