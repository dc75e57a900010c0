"""tern_attention by the kernel and the cluster size that a call takes, on the
GPU against the fp64 oracle: each test asks tern_attention_plan where its
sizes go and says so, so that a change of the rule cannot lead it elsewhere.

Bars.  Tiles: the fp32 bound that the oracle derives with the probabilities
rounded to bf16 once (2^-8 relative).  Rows: the probabilities enter as two
bf16, value and remainder, so 2^-8 of 2^-8 is left.  Then one rounding of the
output.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from bit_post_quantised_b200 import tern
from oracle import block_ops as ref

pytestmark = pytest.mark.gpu
ROWS, TILES = tern.ATTENTION_ROWS, tern.ATTENTION_TILES


def rand(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16)


def inputs(B, Lq, Lk, H, Hkv, D, seed=0, std=1.4):
    s = seed + B + 3 * Lq + 5 * Lk + 7 * H + D
    return (rand((B, Lq, H, D), s, std).cuda(), rand((B, Lk, Hkv, D), s + 1, std).cuda(),
            rand((B, Lk, Hkv, D), s + 2).cuda())


def f64(t):
    return t.detach().cpu().double().numpy()


def close(o, q, k, v, kernel, scale=None, valid=None):
    qd, kd, vd = f64(q), f64(k), f64(v)
    want, av, big = ref.attention(qd, kd, vd, qd.shape[-1] ** -0.5 if scale is None else scale, None,
                                  None if valid is None else valid.numpy())
    e = ref.attention_bound(qd, kd, av, big, ref.BF16 if kernel == TILES else ref.BF16 ** 2)
    got = f64(o)
    bad = ~(np.abs(got - want) <= ref.BF16 * (np.abs(want) + e) + e)
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} out of tolerance, first at {np.argwhere(bad)[0]}"
    assert tern.device_status() == 0


# Sizes, and where they go on a B200 (148 SMs).
EIGHT = [(1, 256, 16384, 4, 4, 128), (1, 256, 16384, 8, 8, 64), (1, 300, 8192, 4, 2, 128), (1, 129, 9001, 5, 5, 96),
         (2, 250, 16001, 3, 3, 40)]
ONE = [(1, 300, 200, 24, 24, 128), (1, 300, 200, 24, 24, 64), (1, 1700, 200, 24, 8, 96)]
SHARED = [(1, 300, 4000, 4, 4, 128), (1, 300, 4000, 4, 4, 64), (1, 1000, 1500, 5, 5, 128)]
FEW = [(1, 1, 512, 24, 24, 128), (2, 1, 17, 6, 2, 64), (3, 17, 531, 16, 4, 64), (1, 40, 700, 8, 4, 128), (1, 1, 5000, 2, 2, 64),
       (2, 129, 257, 3, 3, 128), (1, 255, 64, 2, 1, 40), (1, 7, 2, 4, 4, 64), (1, 3, 9000, 8, 1, 72)]


@pytest.mark.parametrize("B,Lq,Lk,H,Hkv,D", FEW)
@pytest.mark.parametrize("masked", [False, True])
def test_rows_lose_nothing_but_the_last_rounding(B, Lq, Lk, H, Hkv, D, masked):
    q, k, v = inputs(B, Lq, Lk, H, Hkv, D, seed=31)
    assert tern.attention_plan(q, k, v)[0] == ROWS
    if not masked:
        return close(tern.attention(q, k, v), q, k, v, ROWS)
    m = torch.rand(B, Lk, generator=torch.Generator().manual_seed(Lk)) < 0.7
    kd, vd = k.clone(), v.clone()
    kd[(~m).cuda()] = float("inf")
    vd[(~m).cuda()] = float("nan")
    close(tern.attention(q, kd, vd, key_mask=m.cuda()), q, k, v, ROWS, valid=m)


@pytest.mark.parametrize("B,Lq,Lk,H,Hkv,D", EIGHT)
@pytest.mark.parametrize("kind", ["none", "len", "short", "mask"])
def test_eight_ctas_share_the_keys(B, Lq, Lk, H, Hkv, D, kind):
    """Whole lengths, one that ends inside the sixth share, one that leaves
    seven shares without a key, a mask that empties the shares in the middle
    and (with two entries) an entry without a key; rows behind the last query
    as they were; the same bits every time."""
    q, k, v = inputs(B, Lq, Lk, H, Hkv, D, seed=41)
    assert tern.attention_plan(q, k, v) == (TILES, 8)
    n = m = None
    valid = torch.ones(B, Lk, dtype=torch.bool)
    if kind in ("len", "short"):
        n = torch.tensor([Lk * 11 // 16 + 3 if kind == "len" else 77, 0][:B], dtype=torch.int32)
        valid &= torch.arange(Lk)[None] < n[:, None]
    elif kind == "mask":
        m = torch.rand(B, Lk, generator=torch.Generator().manual_seed(Lq)) < 0.5
        m[0, Lk // 4:Lk // 2 + 300] = False
        m[1:] = False
        valid &= m
    bad = (~valid).cuda()
    kd, vd = k.clone(), v.clone()
    kd[bad] = float("nan")
    vd[bad] = float("inf")
    n, m = (None if n is None else n.cuda()), (None if m is None else m.cuda())
    out = torch.full((B, Lq + 2, H, D), 5.0, dtype=torch.bfloat16, device="cuda")
    o = tern.attention(q, kd, vd, kv_len=n, key_mask=m, out=out[:, :Lq])
    close(o, q, k, v, TILES, valid=valid)
    assert (o[~valid.any(1)] == 0).all() and (out[:, Lq:] == 5).all()
    for _ in range(3):
        assert torch.equal(tern.attention(q, kd, vd, kv_len=n, key_mask=m), o)


def test_eight_ctas_on_two_streams_and_in_a_graph():
    a, b = inputs(*EIGHT[0]), inputs(*EIGHT[1])
    assert tern.attention_plan(*a) == (TILES, 8) and tern.attention_plan(*b) == (TILES, 8)
    wa, wb = tern.attention(*a), tern.attention(*b)
    s, r = torch.cuda.Stream(), torch.cuda.Stream()
    for st in (s, r):
        st.wait_stream(torch.cuda.current_stream())
    oa = [tern.attention(*a, stream=s) for _ in range(6)]
    ob = [tern.attention(*b, stream=r) for _ in range(6)]
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
    close(out, *a, TILES)


CASES = [(s, ROWS, None) for s in FEW if s[1] > 1] + [(s, TILES, 1) for s in ONE] + [(s, TILES, None) for s in SHARED] + [
    (s, TILES, 8) for s in EIGHT[:2]]


def goes(q, k, v, kernel, ctas):
    got = tern.attention_plan(q, k, v)
    assert got[0] == kernel and (ctas is None or got[1] == ctas), got
    assert ctas is not None or kernel == ROWS or got[1] > 1, got


@pytest.mark.parametrize("size,kernel,ctas", CASES)
def test_a_nan_score_stays_in_its_row(size, kernel, ctas):
    q, k, v = inputs(*size)
    goes(q, k, v, kernel, ctas)
    want = tern.attention(q, k, v)
    q[0, 1, 0, 3] = float("nan")
    got = tern.attention(q, k, v)
    assert torch.isnan(got[0, 1, 0]).all()
    got[0, 1, 0] = want[0, 1, 0]
    assert torch.equal(got, want)


def lone(q, k, key, value):
    """Query 1 and `key` meet in one channel, with the product |value| * value;
    every other score of either is zero."""
    q[0, 1], k[0, key] = 0.0, 0.0
    q[0, :, :, 3] = 0.0
    k[0, :, :, 3] = 0.0
    q[0, 1, :, 3] = abs(value)
    k[0, key, :, 3] = value


@pytest.mark.parametrize("size,kernel,ctas", CASES)
def test_a_scaled_score_that_overflows_gives_nan_rows(size, kernel, ctas):
    """2^60 * 2^60 * 2^40 = 2^160: not in fp32.  The other rows are finite."""
    q, k, v = inputs(*size)
    goes(q, k, v, kernel, ctas)
    lone(q, k, size[2] // 2, 2.0 ** 60)
    got = tern.attention(q, k, v, scale=2.0 ** 40)
    assert torch.isnan(got[0, 1]).all()
    rest = torch.arange(size[1], device="cuda") != 1
    assert torch.isfinite(got[0, rest]).all() and torch.isfinite(got[1:]).all()
    assert tern.device_status() == 0


@pytest.mark.parametrize("size,kernel,ctas", [((1, 4, 300, 1, 1, 64), ROWS, None), ((1, 300, 300, 24, 24, 128), TILES, 1),
                                              ((1, 300, 300, 24, 24, 64), TILES, 1), ((1, 1000, 300, 24, 24, 128), TILES, 1)])
def test_keys_behind_32_bit_offsets(size, kernel, ctas):
    """Keys and values whose tokens span more than 2^32 bytes of one buffer."""
    _, Lq, Lk, H, _, D = size
    ld = 1 << 24
    big = torch.empty(Lk * ld, dtype=torch.bfloat16, device="cuda")
    k, v = (big[i * H * D:].as_strided((1, Lk, H, D), (0, ld, D, 1)) for i in range(2))
    q, kk, vv = inputs(*size)
    goes(q, k, v, kernel, ctas)
    k.copy_(kk)
    v.copy_(vv)
    assert torch.equal(tern.attention(q, k, v), tern.attention(q, kk, vv))


@pytest.mark.parametrize("size,kernel,ctas", CASES)
@pytest.mark.parametrize("scale", [2.0 ** 16, 2.0 ** 27, 2.0 ** 100])
def test_scaled_scores_far_from_zero(size, kernel, ctas, scale):
    """A scale by which only the row's highest score counts (or several, where
    they are equal): q and k hold small whole numbers, so that scores are
    exact in fp32 and ties are ties."""
    B, Lq, Lk, H, Hkv, D = size
    g = torch.Generator().manual_seed(Lk + H)
    q = torch.randint(-3, 4, (B, Lq, H, D), generator=g).to(torch.bfloat16).cuda()
    k = torch.randint(-3, 4, (B, Lk, Hkv, D), generator=g).to(torch.bfloat16).cuda()
    v = rand((B, Lk, Hkv, D), 3).cuda()
    goes(q, k, v, kernel, ctas)
    got = f64(tern.attention(q, k, v, scale=scale))
    G = H // Hkv
    qd, kd, vd = q.double().cpu(), k.double().cpu().repeat_interleave(G, 2), v.double().cpu().repeat_interleave(G, 2)
    s = torch.einsum("bqhd,bkhd->bhqk", qd, kd)
    p = (s == s.amax(-1, keepdim=True)).double()
    p /= p.sum(-1, keepdim=True)
    want = torch.einsum("bhqk,bkhd->bqhd", p, vd).numpy()
    av = torch.einsum("bhqk,bkhd->bqhd", p, vd.abs()).numpy()
    # Equal scores have equal probabilities, exactly 1 against their maximum or 2^(up to 8 and its
    # rounding, 2^-20) against an older reference, rounded alike: the factor's bf16 rounding stays.
    e = ((ref.BF16 if kernel == TILES else ref.BF16 ** 2) + 2.0 ** -20 + (Lk / 4 + 16) * ref.F32) * av
    assert np.all(np.abs(got - want) <= ref.BF16 * (np.abs(want) + e) + e)
    assert tern.device_status() == 0


def masked_like(q, k, v, gone, scale):
    """fp64 attention of entry 0 without the keys `gone`."""
    keep = ~gone.cpu()
    return ref.attention(f64(q[:1]), f64(k[:1]), f64(v[:1]), scale, None, keep[None].numpy())


@pytest.mark.parametrize("size,kernel,ctas", CASES)
@pytest.mark.parametrize("raw", [True, False])
def test_rows_whose_scores_are_all_minus_infinity(size, kernel, ctas, raw):
    """Query 1's scores with every key are -inf, from an infinite channel or from
    the scale (-2^60 * 2^60 * 2^40): NaN, as a maximum that is not finite gives.
    The others' are as they are without that channel."""
    B, Lq, Lk, H, Hkv, D = size
    q, k, v = inputs(*size)
    goes(q, k, v, kernel, ctas)
    scale = D ** -0.5 if raw else 2.0 ** 40
    q[0, :, :, 3] = 0.0
    k[0, :, :, 3] = 1.0 if raw else -2.0 ** 60
    if not raw:
        q[0, 1] = 0.0
    q[0, 1, :, 3] = float("-inf") if raw else 2.0 ** 60
    got = tern.attention(q, k, v, scale=scale)
    assert torch.isnan(got[0, 1]).all()
    rest = torch.arange(Lq, device="cuda") != 1
    assert torch.isfinite(got[0, rest]).all() and torch.isfinite(got[1:]).all()
    if raw:
        q[0, 1, :, 3] = 0.0
        want = tern.attention(q, k, v, scale=scale)
        assert torch.equal(got[0, rest], want[0, rest]) and torch.equal(got[1:], want[1:])


QUARTERS = [c for c in CASES if c[0][2] >= 8]  # keys enough for a quarter of them


@pytest.mark.parametrize("size,kernel,ctas", QUARTERS)
@pytest.mark.parametrize("raw", [True, False])
@pytest.mark.parametrize("where", ["first", "last"])
def test_keys_at_minus_infinity_before_and_behind_finite_ones(size, kernel, ctas, raw, where):
    """Three quarters of the keys score -inf with every query, raw or by the
    scale; the rest decide, as if those keys were not there."""
    B, Lq, Lk, H, Hkv, D = size
    q, k, v = inputs(*size)
    goes(q, k, v, kernel, ctas)
    gone = torch.arange(Lk, device="cuda") < Lk - Lk // 4
    if where == "last":
        gone = gone.flip(0)
    scale = D ** -0.5 if raw else 2.0 ** 40
    if not raw:  # 2^40 * 2^-20 * 2^-20 of the scores: ordinary sizes
        q, k = q * 2.0 ** -20, k * 2.0 ** -20
        q[0, :, :, 3], k[0, :, :, 3] = 2.0 ** 60, 0.0
        k[0, gone, :, 3] = -2.0 ** 60
    else:
        q[0, :, :, 3], k[0, :, :, 3] = 1.0, 0.0
        k[0, gone, :, 3] = float("-inf")
    got = f64(tern.attention(q, k, v, scale=scale)[:1])
    k[0, gone, :, 3] = 0.0
    want, av, big = masked_like(q, k, v, gone, scale)
    e = ref.attention_bound(f64(q[:1]), f64(k[:1]), av, big, ref.BF16 if kernel == TILES else ref.BF16 ** 2)
    assert np.all(np.abs(got - want) <= ref.BF16 * (np.abs(want) + e) + e)


@pytest.mark.parametrize("size,kernel,ctas", QUARTERS)
def test_minus_infinity_under_a_mask(size, kernel, ctas):
    """The valid keys score -inf, the masked ones would not: NaN rows; an entry
    without a valid key is zeros beside them."""
    B, Lq, Lk, H, Hkv, D = size
    q, k, v = inputs(2, *size[1:])
    m = torch.zeros(2, Lk, dtype=torch.bool, device="cuda")
    m[0, Lk // 2:Lk // 2 + Lk // 4] = True
    q[0, :, :, 3], k[0, :, :, 3] = 1.0, 0.0
    k[0, m[0], :, 3] = float("-inf")
    got = tern.attention(q, k, v, key_mask=m)
    assert torch.isnan(got[0]).all() and (got[1] == 0).all()
    n = torch.tensor([Lk // 4, 0], dtype=torch.int32, device="cuda")
    k[0, :, :, 3] = 0.0
    k[0, :Lk // 4, :, 3] = float("-inf")
    got = tern.attention(q, k, v, kv_len=n)
    assert torch.isnan(got[0]).all() and (got[1] == 0).all()
    assert tern.device_status() == 0


@pytest.mark.parametrize("Lk", [1, 3])
def test_more_than_2_to_the_31_query_rows(Lk):
    """2^28 + 5 queries of 8 heads of 8 channels (34 GB of output): with one key
    every output is that key's value; with three, stretches at the ends and
    around the offsets of 2^31 and 2^32 elements against fp64."""
    Lq, H, D = (1 << 28) + 5, 8, 8
    g = torch.Generator(device="cuda").manual_seed(Lk)
    q = torch.randn(1, Lq, 1, D, generator=g, device="cuda", dtype=torch.bfloat16).expand(1, Lq, H, D)
    k, v = (torch.randn(1, Lk, H, D, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    out = torch.full((1, Lq + 1, H, D), 3.0, dtype=torch.bfloat16, device="cuda")
    try:
        o = tern.attention(q, k, v, out=out[:, :Lq])
        assert (out[:, Lq] == 3).all() and tern.device_status() == 0
        if Lk == 1:
            for at in range(0, Lq, 1 << 24):
                assert (o[:, at:at + (1 << 24)] == v).all()
            return
        kernel = tern.attention_plan(q, k, v)[0]
        for at in (0, (1 << 25) - 500, (1 << 26) - 500, (1 << 27) + 77, Lq - 1000):
            close(o[:, at:at + 1000], q[:, at:at + 1000], k, v, kernel)
    finally:
        del out, q
        o = None
        torch.cuda.empty_cache()


@pytest.mark.parametrize("B,L,H,D", [(2, 9, 4, 64), (1, 700, 24, 128)])
def test_output_between_its_inputs(B, L, H, D):
    """o, q, k and v side by side in every head of one tensor."""
    z = rand((B, L, H, 4, D), 1, 1.4).cuda()
    q, k, v, o = (z[:, :, :, i] for i in range(4))
    old = z.clone()
    kernel = tern.attention_plan(q, k, v)[0]
    assert kernel == (TILES if L == 700 else ROWS)
    close(tern.attention(q, k, v, out=o), q, k, v, kernel)
    assert torch.equal(z[:, :, :, :3], old[:, :, :, :3])
