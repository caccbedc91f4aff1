"""The bf16 softmax kernels where every block walks several items: item slots and row
buffers that are used again, barrier phases that come round, groups and teams that
hand over from one item to the next.  Against float64, head by head."""
import pytest
import torch

from tests import softmax_ref as ref
from tests.test_softmax_attn_gpu import BF16, TYPES, draw

pytestmark = pytest.mark.gpu


def plan(B, Hq, Hk, Lq, Lk, W, causal):
    """Row tiles per item, and items per SM of the forward, the query and the key sweep
    (the launch rules of softmax_attn.cu)."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    nq = 128 // (Hq // Hk)
    tiles, W = B * Hk * -(-Lq // nq), min(W, Lk)
    nr = 1 if tiles <= sms else 4 if W >= 4096 and tiles >= 6 * sms else 2
    items = B * Hk * -(-Lq // (nr * nq))
    if items < sms:
        chunks = -(-min(Lk, W + (0 if causal else W) + nr * nq) // 64)
        items *= max(1, min(2 * sms // items, chunks // 8))
    return nr, items / sms, tiles / sms, B * Hk * -(-Lk // 128) / sms


def check_heads(q, k, v, dO, *, mask=None, q_pos=None, eps=1.0, **kw):
    import banded_log_domain_b200 as sa

    B, Hq, Hk = q.shape[0], q.shape[1], k.shape[1]
    G, dt = Hq // Hk, q.dtype
    o, u = sa.sinkhorn_attn_softmax_fwd(q, k, v, eps=eps, mask=mask, q_pos=q_pos, **kw)
    got = sa.sinkhorn_attn_softmax_bwd(q, k, v, o, dO, u, eps=eps, mask=mask, q_pos=q_pos, **kw)
    for b in range(B):
        bb = slice(b, b + 1)
        one = dict(kw, eps=eps, mask=None if mask is None else mask[bb], q_pos=None if q_pos is None else q_pos[bb])
        for h in range(Hk):
            hq, hk = slice(G * h, G * h + G), slice(h, h + 1)
            x = (q[bb, hq], k[bb, hk], v[bb, hk], dO[bb, hq])
            wo, wu, P = ref.forward(*x[:3], **one)
            lim = ref.bounds(*x, P, dt, eps=eps)
            ref.close(f"o of sequence {b}, head {h}", o[bb, hq], wo, lim["o"], dt)
            assert float((u[bb, hq].double() - wu).abs().max()) <= ref.U_ATOL
            for n, y, s, w in zip(("dq", "dk", "dv"), got, (hq, hk, hk), ref.backward(*x, P, eps=eps)):
                ref.close(f"{n} of sequence {b}, head {h}", y[bb, s], w, lim[n], dt)


# (B, Hq, Hk, Lq, Lk, W), row tiles per item, items per SM at least: forward and sweeps
SHAPES = [
    ((4, 16, 16, 3600, 3600, 100), 2, 6, 6, 6),
    ((3, 21, 7, 4000, 4000, 130), 2, 6, 12, 4),    # tiles of 126 of 128 rows
    ((7, 16, 16, 4101, 4101, 4101), 4, 6, 24, 24),
    ((4, 28, 4, 4099, 4099, 4097), 4, 6, 24, 3),   # tiles of 126 rows; 7 heads to a key item
    ((1, 50, 50, 256, 4000, 4000), 1, 1.3, 0.6, 10),  # keys in two parts
    ((8, 16, 8, 1500, 3000, 700), 2, 5, 10, 10),  # a piece of a prompt
]


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("masked", [None, "tail", "holes"])
@pytest.mark.parametrize("shape,nr,fwd,dq,dkv", SHAPES)
def test_several_items_per_block(shape, nr, fwd, dq, dkv, masked, causal):
    B, Hq, Hk, Lq, Lk, W = shape
    p = plan(*shape, causal)
    assert p[0] == nr and p[1] >= fwd and p[2] >= dq and p[3] >= dkv, p
    q, k, v, dO = draw(BF16, B, Hq, Hk, Lq, Lk, seed=Lk)
    g = torch.Generator("cuda").manual_seed(W)
    mask = None
    if masked == "tail":
        n = torch.randint(Lk // 3, Lk + 1, (B, 1), generator=g, device="cuda")
        mask = (torch.arange(Lk, device="cuda")[None] < n).to(torch.uint8)
    elif masked == "holes":
        mask = (torch.rand(B, Lk, generator=g, device="cuda") < 0.8).to(torch.uint8)
        mask[:, Lk // 2:Lk // 2 + 200] = 0  # chunks without a key
    q_pos = None
    if Lq < Lk:  # from the first tokens to the last
        q_pos = torch.linspace(0, Lk - Lq, B, device="cuda").round().to(torch.int32)
    check_heads(q, k, v, dO, W=W, causal=causal, mask=mask, q_pos=q_pos)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,G,Lq", [(64, 4, 1), (65, 4, 1), (130, 1, 1), (8, 8, 2), (8, 8, 3), (3, 5, 4)])
def test_many_sequences_and_rows_of_new_tokens(dtype, B, G, Lq):
    # either side of the single-token kernel's limits on sequences and rows
    Lk = 700
    q, k, v, dO = draw(dtype, B, 2 * G, 2, Lq, Lk, seed=B)
    q_pos = torch.randint(0, Lk - Lq + 1, (B,), generator=torch.Generator("cuda").manual_seed(G), device="cuda",
                          dtype=torch.int32)
    check_heads(q, k, v, dO, W=Lk, causal=True, q_pos=q_pos)
    check_heads(q, k, v, dO, W=90, causal=True, q_pos=q_pos)
