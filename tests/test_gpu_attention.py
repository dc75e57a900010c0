"""tern_attention against the fp64 oracle on the GPU.

Bar: the fp32 bound that the oracle derives (scores, exponentials, sums, and
2^-8 relative for the probabilities' rounding to bf16 as the tensor cores'
operand), then one rounding of the output to bf16.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from bit_post_quantised_b200 import tern
from oracle import block_ops as ref

pytestmark = pytest.mark.gpu


def rand(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16)


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def close(o, q, k, v, scale=None, kv_len=None, key_mask=None):
    qd, kd, vd = f64(q), f64(k), f64(v)
    if qd.ndim == 3:
        qd, kd, vd = qd[None], kd[None], vd[None]
        key_mask = None if key_mask is None else key_mask[None]
    want, av, big = ref.attention(qd, kd, vd, qd.shape[-1] ** -0.5 if scale is None else scale,
                                  None if kv_len is None else kv_len.cpu().numpy(),
                                  None if key_mask is None else key_mask.cpu().numpy())
    e = ref.attention_bound(qd, kd, av, big, ref.BF16)
    got = f64(o).reshape(want.shape)
    bad = ~(np.abs(got - want) <= ref.BF16 * (np.abs(want) + e) + e)
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} out of tolerance, first at {np.argwhere(bad)[0]}"
    assert tern.device_status() == 0


def inputs(B, Lq, Lk, H, Hkv, D, seed=0, std=1.4):
    s = seed + B + 3 * Lq + 5 * Lk + 7 * H + D
    return (rand((B, Lq, H, D), s, std).cuda(), rand((B, Lk, Hkv, D), s + 1, std).cuda(),
            rand((B, Lk, Hkv, D), s + 2).cuda())


SIZES = [(1, 1, 1, 1, 1, 8), (1, 1, 1, 1, 1, 128), (1, 1, 512, 24, 24, 128), (2, 1, 17, 6, 2, 64), (1, 1, 5000, 2, 2, 64),
         (3, 17, 531, 16, 4, 64), (2, 3, 33, 8, 1, 72), (1, 16, 127, 4, 4, 96), (1, 15, 128, 3, 3, 80),
         (2, 64, 129, 4, 2, 128), (1, 127, 255, 2, 2, 128), (1, 128, 256, 2, 2, 64), (2, 129, 257, 3, 3, 128),
         (1, 255, 64, 2, 1, 40), (1, 256, 128, 2, 2, 128), (1, 257, 1, 2, 2, 128), (1, 385, 640, 4, 2, 64),
         (1, 1000, 77, 5, 5, 120), (2, 300, 1030, 2, 2, 128), (1, 513, 384, 1, 1, 16)]
# Enough query rows for the tile kernel: odd and whole tiles, one key tile or many, one query tile in the last pair,
# grouped heads, more units than SMs.
TILES = [(2, 129, 257, 12, 12, 128), (1, 257, 300, 12, 3, 64), (1, 384, 128, 16, 16, 128), (3, 128, 64, 20, 10, 72),
         (1, 1300, 65, 12, 12, 96), (1, 2049, 640, 2, 2, 128), (1, 700, 1, 40, 40, 64), (2, 300, 1030, 10, 5, 128),
         (1, 4200, 96, 20, 20, 8), (1, 640, 129, 70, 70, 128)]


@pytest.mark.parametrize("B,Lq,Lk,H,Hkv,D", SIZES + TILES)
def test_matches_oracle(B, Lq, Lk, H, Hkv, D):
    q, k, v = inputs(B, Lq, Lk, H, Hkv, D)
    close(tern.attention(q, k, v), q, k, v)


@pytest.mark.parametrize("B,Lq,Lk,H,Hkv,D", [s for s in SIZES if s[2] > 1] + [s for s in TILES[:8] if s[2] > 1])
@pytest.mark.parametrize("kind", ["len", "mask", "both"])
def test_masked_keys(B, Lq, Lk, H, Hkv, D, kind):
    """Lengths of zero, one, a part and beyond the end, holes, entries without
    a key; masked keys and values hold infinities and NaN."""
    B = 5
    q, k, v = inputs(B, Lq, Lk, H, Hkv, D, seed=9)
    g = torch.Generator().manual_seed(Lk)
    n = torch.tensor([Lk // 3, 0, 1, Lk + 7, -2], dtype=torch.int32)
    m = torch.rand(B, Lk, generator=g) < 0.6
    m[3] = False
    m[4, :] = False
    m[4, Lk - 1] = True
    n, m = (n if kind != "mask" else None), (m if kind != "len" else None)
    valid = torch.ones(B, Lk, dtype=torch.bool)
    if n is not None:
        valid &= torch.arange(Lk)[None] < n[:, None]
    if m is not None:
        valid &= m
    kd, vd = k.clone(), v.clone()
    bad = (~valid).cuda()
    kd[bad] = float("nan")
    vd[bad] = float("inf")
    vd[:, ::2][bad[:, ::2]] = float("nan")
    n, m = (None if n is None else n.cuda()), (None if m is None else m.cuda())
    o = tern.attention(q, kd, vd, kv_len=n, key_mask=m)
    close(o, q, k, v, kv_len=n, key_mask=m)
    assert (o[~valid.any(1)] == 0).all()


def test_no_keys_no_queries():
    q, k, v = inputs(2, 5, 0, 4, 2, 64)
    assert (tern.attention(q, k, v) == 0).all()
    q, k, v = inputs(2, 300, 0, 4, 2, 128)
    assert (tern.attention(q, k, v) == 0).all()
    q, k, v = inputs(2, 0, 5, 4, 2, 64)
    assert tern.attention(q, k, v).shape == (2, 0, 4, 64)


@pytest.mark.parametrize("Lq,Lk", [(5, 40), (300, 260), (900, 140)])
def test_layouts(Lq, Lk):
    """Slices of fused projections, heads-first tensors, a broadcast of the
    keys over the batch, an output slice whose surroundings stay as they were,
    no batch dimension, a mask that is a view."""
    B, H, D = 2, 4, 64
    z = rand((B, Lq, 3 * H * D + 8), 1).cuda()
    q = z[..., 8:8 + H * D].view(B, Lq, H, D)
    kv = rand((1, Lk, 2 * H * D), 2).cuda()
    k, v = (t.view(1, Lk, H, D).expand(B, Lk, H, D) for t in (kv[..., :H * D], kv[..., H * D:]))
    out = torch.full((B, Lq + 1, 2 * H * D), 3.0, dtype=torch.bfloat16, device="cuda")
    o = tern.attention(q, k, v, out=out[:, :Lq, H * D:].view(B, Lq, H, D))
    close(o, q, k, v)
    assert (out[:, :, :H * D] == 3).all() and (out[:, Lq] == 3).all()
    qh, kh, vh = (rand((B, H, n, D), i).cuda().transpose(1, 2) for i, n in ((3, Lq), (4, Lk), (5, Lk)))
    mask = (torch.arange(B * 2 * Lk, device="cuda").view(B, 2 * Lk) % 5 != 0)[:, Lk:]
    oh = torch.empty(B, H, Lq, D, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    close(tern.attention(qh, kh, vh, key_mask=mask, out=oh), qh, kh, vh, key_mask=mask)
    # without a batch dimension; not bit for bit the batch's, whose size has a say in how the keys are split
    close(tern.attention(qh[0], kh[0], vh[0], key_mask=mask[0]), qh[0], kh[0], vh[0], key_mask=mask[0])


@pytest.mark.parametrize("Lq,Lk", [(3, 100), (200, 300), (1300, 300)])
def test_scales_and_peaked_scores(Lq, Lk):
    """Scores of hundreds, growing along the keys (each tile raises the
    maximum) and falling; a scale of its own."""
    q, k, v = inputs(1, Lq, Lk, 2, 2, 128, std=3.0)
    up = torch.linspace(-4, 4, Lk, device="cuda")[None, :, None, None]
    for kk in (k, (k.float() + up * q.float().mean(1, keepdim=True)).bfloat16(),
               (k.float() - up * q.float().mean(1, keepdim=True)).bfloat16()):
        for scale in (0.5, 0.01):
            close(tern.attention(q, kk, v, scale=scale), q, kk, v, scale=scale)


@pytest.mark.parametrize("Lq", [2, 300, 1700])
def test_scores_that_are_not_finite_stay_in_their_rows(Lq):
    q, k, v = inputs(1, Lq, 200, 2, 2, 64)
    want = tern.attention(q, k, v)
    q[0, 1, 0, 3] = float("nan")
    got = tern.attention(q, k, v)
    assert torch.isnan(got[0, 1, 0]).all()
    got[0, 1, 0] = want[0, 1, 0]
    assert torch.equal(got, want)


@pytest.mark.parametrize("Lq,Lk", [(4, 300), (260, 300), (2300, 300)])
def test_behind_32_bit_offsets(Lq, Lk):
    """Keys and values more than 2^32 bytes apart in one buffer."""
    D, ld = 64, 1 << 24
    big = torch.empty(Lk * ld, dtype=torch.bfloat16, device="cuda")
    k, v = big.as_strided((1, Lk, 1, D), (0, ld, D, 1)), big[D:].as_strided((1, Lk, 1, D), (0, ld, D, 1))
    q, kk, vv = inputs(1, Lq, Lk, 1, 1, D)
    k.copy_(kk)
    v.copy_(vv)
    assert torch.equal(tern.attention(q, k, v), tern.attention(q, kk, vv))


@pytest.mark.parametrize("Lq,Lk,H", [(1, 700, 8), (40, 700, 8), (520, 300, 2), (1030, 700, 12)])
def test_same_call_same_bits_other_stream_and_graph(Lq, Lk, H):
    q, k, v = inputs(2, Lq, Lk, H, H // 2, 128)
    n = torch.tensor([Lk, Lk // 2], dtype=torch.int32, device="cuda")
    want = tern.attention(q, k, v, kv_len=n)
    for _ in range(5):
        assert torch.equal(tern.attention(q, k, v, kv_len=n), want)
    s = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for st in s:
        st.wait_stream(torch.cuda.current_stream())
        outs += [tern.attention(q, k, v, kv_len=n, stream=st) for _ in range(3)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    out = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tern.attention(q, k, v, kv_len=n, out=out)
    n.copy_(torch.tensor([3, Lk], dtype=torch.int32))
    q.copy_(rand(q.shape, 77))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, tern.attention(q, k, v, kv_len=n))
    close(out, q, k, v, kv_len=n)


def test_broadcast_tokens():
    """Keys and values that are one row for every token (stride 0), and queries likewise."""
    q, k, v = inputs(1, 1200, 300, 4, 4, 64)
    k1, v1, q1 = k[:, :1].expand(1, 300, 4, 64), v[:, :1].expand(1, 300, 4, 64), q[:, :1].expand(1, 1200, 4, 64)
    close(tern.attention(q, k1, v1), q, k1, v1)
    close(tern.attention(q1, k, v), q1, k, v)


def test_two_streams_at_once():
    """Two calls in flight together, rows and tiles, each on its own inputs."""
    a, b = inputs(1, 17, 1531, 16, 4, 64), inputs(1, 2049, 640, 4, 4, 128)
    wa, wb = tern.attention(*a), tern.attention(*b)
    s, r = torch.cuda.Stream(), torch.cuda.Stream()
    for st in (s, r):
        st.wait_stream(torch.cuda.current_stream())
    oa = [tern.attention(*a, stream=s) for _ in range(8)]
    ob = [tern.attention(*b, stream=r) for _ in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, wa) for o in oa) and all(torch.equal(o, wb) for o in ob)
    assert tern.device_status() == 0


def test_units_longer_than_the_wait_limit():
    """The limit bounds waits that make no progress: a unit of many keys may
    take longer than it (200 key tiles, some 300 us; heads of two query tiles and of one)."""
    q, k, v = inputs(1, 300, 25600, 80, 5, 64)
    want = tern.attention(q, k, v)
    torch.cuda.synchronize()
    tern.set_wait_limit_ns(50_000)
    try:
        got = tern.attention(q, k, v)
        assert tern.device_status() == 0
    finally:
        tern.set_wait_limit_ns(1_000_000_000)
    assert torch.equal(got, want)


@pytest.mark.parametrize("Lq", [2, 300, 1700])
def test_scaled_scores_that_overflow_give_nan_rows(Lq):
    """Finite scores whose product with the scale is not: their rows are NaN, the others as before."""
    q, k, v = inputs(1, Lq, 200, 2, 2, 64)
    q[0, 1], k[0, 5] = 0.0, 0.0
    want = tern.attention(q, k, v, scale=2.0 ** 40)
    q[0, 1, :, 3] = 2.0 ** 60
    k[0, 5, :, 3] = 2.0 ** 60
    k[0, :5, :, 3] = 0.0
    k[0, 6:, :, 3] = 0.0
    q[0, 0, :, 3] = 0.0
    q[0, 2:, :, 3] = 0.0
    got = tern.attention(q, k, v, scale=2.0 ** 40)
    assert torch.isnan(got[0, 1]).all()
    rest = torch.arange(Lq, device="cuda") != 1
    assert torch.isfinite(got[0, rest]).all() and torch.isfinite(want).all()


@pytest.mark.parametrize("Lq,Lk,D", [(300, 200, 128), (300, 129, 64), (129, 400, 96), (513, 64, 128)])
def test_many_units_with_empty_entries(Lq, Lk, D):
    """Several units a CTA: of one query tile and of two, of no, one and more key tiles in turn."""
    B, H = 13, 12
    q, k, v = inputs(B, Lq, Lk, H, H, D, seed=3)
    n = torch.tensor([0, Lk, 1, 0, 0, 127, 128, 129, 0, Lk, 5, Lk - 1, 0], dtype=torch.int32)
    valid = torch.arange(Lk)[None] < n[:, None]
    k[(~valid).cuda()] = float("nan")
    v[(~valid).cuda()] = float("inf")
    out = torch.full((B, Lq + 3, H, D), 9.0, dtype=torch.bfloat16, device="cuda")
    o = tern.attention(q, k, v, kv_len=n.cuda(), out=out[:, :Lq])
    k[(~valid).cuda()] = 0.0
    v[(~valid).cuda()] = 0.0
    close(o, q, k, v, kv_len=n)
    assert (o[n == 0] == 0).all() and (out[:, Lq:] == 9).all()


@pytest.mark.parametrize("B,Lq,Lk,H,Hkv,D", [(1, 256, 2700, 8, 8, 128), (1, 513, 2049, 4, 2, 96), (2, 300, 4000, 6, 3, 64),
                                             (1, 1000, 1500, 5, 5, 40), (1, 129, 3333, 40, 40, 128), (3, 257, 1025, 8, 8, 128)])
@pytest.mark.parametrize("kind", ["none", "len", "mask"])
def test_few_units_of_many_keys(B, Lq, Lk, H, Hkv, D, kind):
    """A cluster shares the keys of a unit: shares without a key, ends inside a
    tile, NaN and infinities in masked places, entries without a key, the
    rows behind the last one as they were."""
    if kind != "none":
        B = 3
    q, k, v = inputs(B, Lq, Lk, H, Hkv, D, seed=21)
    n = m = None
    valid = torch.ones(B, Lk, dtype=torch.bool)
    if kind == "len":
        n = torch.tensor([Lk // 2 + 3, 0, 130], dtype=torch.int32)
        valid &= torch.arange(Lk)[None] < n[:, None]
    elif kind == "mask":
        m = torch.rand(B, Lk, generator=torch.Generator().manual_seed(Lq)) < 0.5
        m[1, : Lk // 2] = False
        m[2] = False
        valid &= m
    bad = (~valid).cuda()
    kd, vd = k.clone(), v.clone()
    kd[bad] = float("nan")
    vd[bad] = float("inf")
    n, m = (None if n is None else n.cuda()), (None if m is None else m.cuda())
    out = torch.full((B, Lq + 2, H, D), 5.0, dtype=torch.bfloat16, device="cuda")
    o = tern.attention(q, kd, vd, kv_len=n, key_mask=m, out=out[:, :Lq])
    close(o, q, k, v, kv_len=n, key_mask=m)
    assert (o[~valid.any(1)] == 0).all() and (out[:, Lq:] == 5).all()
    for _ in range(3):
        assert torch.equal(tern.attention(q, kd, vd, kv_len=n, key_mask=m), o)


def test_shared_keys_on_two_streams_and_in_a_graph():
    """Clusters that share a unit's keys: two such calls in flight together, a captured one replayed on new inputs."""
    a, b = inputs(1, 256, 4608, 8, 8, 128), inputs(2, 300, 4000, 6, 3, 64)
    wa, wb = tern.attention(*a), tern.attention(*b)
    s, r = torch.cuda.Stream(), torch.cuda.Stream()
    for st in (s, r):
        st.wait_stream(torch.cuda.current_stream())
    oa = [tern.attention(*a, stream=s) for _ in range(8)]
    ob = [tern.attention(*b, stream=r) for _ in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, wa) for o in oa) and all(torch.equal(o, wb) for o in ob)
    out = torch.empty_like(wa)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tern.attention(*a, out=out)
    a[0].copy_(rand(a[0].shape, 5))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, tern.attention(*a))
    close(out, *a)


def test_shared_keys_with_peaks_and_scores_that_are_not_finite():
    q, k, v = inputs(1, 300, 4000, 4, 4, 128, std=3.0)
    up = torch.linspace(-4, 4, 4000, device="cuda")[None, :, None, None]
    for kk in ((k.float() + up * q.float().mean(1, keepdim=True)).bfloat16(),
               (k.float() - up * q.float().mean(1, keepdim=True)).bfloat16()):
        close(tern.attention(q, kk, v, scale=0.5), q, kk, v, scale=0.5)
    want = tern.attention(q, k, v)
    q[0, 1, 0, 3] = float("nan")
    got = tern.attention(q, k, v)
    assert torch.isnan(got[0, 1, 0]).all()
    got[0, 1, 0] = want[0, 1, 0]
    assert torch.equal(got, want)
