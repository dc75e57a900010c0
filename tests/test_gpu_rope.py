"""tern_rope_table and tern_rope against the fp64 oracle on the GPU.

Bars.  Table: one rounding to fp32 (2^-24 relative), the 64-bit angle's own
error (2^-50 of it) and the polynomials' truncation (below 1e-11).  Rotation:
fp32 products and sum (4 half steps of |a| + |b|), then one rounding to bf16
(2^-8 relative).
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from bit_post_quantised_b200 import flux, tern
from oracle import block_ops as ref

pytestmark = pytest.mark.gpu


def rand(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(torch.bfloat16)


def f64(t):
    return t.detach().cpu().double().numpy()


def table_close(cs, ids, axes, theta):
    ang = ref.rope_angles(ids.numpy(), axes, theta)
    want = ref.rope_table(ids.numpy(), axes, theta)
    tol = ref.F32 * np.abs(want) + (np.abs(ang) * 2.0 ** -50)[..., None] + 1e-11
    assert np.all(np.abs(f64(cs) - want) <= tol)


def turned_close(y, x, cs, halves):
    xd, c = f64(x), f64(cs)
    want = ref.rope(xd, c, halves)
    P = c.shape[-2]
    mag = np.abs(xd).copy()
    if halves:
        mag[..., :P] += np.abs(xd[..., P:2 * P])
        mag[..., P:2 * P] = mag[..., :P]
    else:
        mag[..., 0:2 * P:2] += np.abs(xd[..., 1:2 * P:2])
        mag[..., 1:2 * P:2] = mag[..., 0:2 * P:2]
    d = 4 * ref.F32 * mag
    assert np.all(np.abs(f64(y) - want) <= ref.BF16 * (np.abs(want) + d) + d)
    assert np.array_equal(f64(y)[..., 2 * P:], xd[..., 2 * P:])


@pytest.mark.parametrize("L,axes,theta", [(1, (2,), 10000.0), (88, (16, 56, 56), 10000.0), (257, (44, 42, 42), 10000.0),
                                          (1000, (6, 2, 90, 30), 1.5), (33, (256,), 1e6), (5, (126, 2), 0.5),
                                          (4099, (64,), 256.0)])
def test_table_matches_oracle(L, axes, theta):
    g = torch.Generator().manual_seed(L)
    ids = torch.randint(-50, 5000, (L, len(axes)), generator=g).float()
    cs = tern.rope_table(ids.cuda(), axes, theta)
    table_close(cs.cpu(), ids, axes, theta)


def test_table_of_far_and_fractional_positions():
    ids = torch.tensor([[0.0, 0.5], [16777215.0, -16777216.0], [1e6 + 0.25, 1 / 3], [-0.0, 123456.75]])
    cs = tern.rope_table(ids.cuda(), (48, 16))
    table_close(cs.cpu(), ids, (48, 16), 10000.0)


def test_table_of_positions_that_are_not_finite():
    ids = torch.tensor([[float("inf"), 1.0], [2.0, float("nan")], [3.0, 4.0]])
    cs = tern.rope_table(ids.cuda(), (4, 4)).cpu()
    assert torch.isnan(cs[0, :2]).all() and torch.isnan(cs[1, 2:]).all()
    assert torch.isfinite(cs[0, 2:]).all() and torch.isfinite(cs[1, :2]).all() and torch.isfinite(cs[2]).all()


def test_table_is_the_one_of_the_block_forward():
    """The linears' rope_cs: within one fp32 step of the table flux.py builds with torch."""
    g = torch.Generator().manual_seed(3)
    ids = torch.randint(0, 64, (88, 3), generator=g).float().cuda()
    cos, sin = flux.rope_cos_sin(ids)
    got = tern.rope_table(ids, (16, 56, 56))
    want = torch.stack([cos, sin], -1)
    assert torch.all((got - want).abs() <= 2.0 ** -23 * want.abs())


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("L,heads,D,axes", [(1, (1,), 16, (16,)), (88, (2, 2), 128, (16, 56, 56)),
                                            (37, (24, 24), 128, (44, 42, 42)), (130, (5, 1), 80, (16, 32, 32)),
                                            (19, (3, 3, 1, 2), 96, (32, 16)), (7, (40, 8), 256, (64, 96, 96)),
                                            (65, (12, 4), 72, (32, 32))])
def test_rope_matches_oracle(L, heads, D, axes, halves):
    g = torch.Generator().manual_seed(L + D)
    ids = torch.randint(0, 300, (L, len(axes)), generator=g).float().cuda()
    cs = tern.rope_table(ids, axes)
    xs = [rand((L, h, D), 10 * i + L).cuda() for i, h in enumerate(heads)]
    keep = [x.clone() for x in xs]
    ys = tern.rope(xs, cs, halves=halves)
    for x, y, k in zip(xs, ys, keep):
        assert torch.equal(x, k)
        turned_close(y, x, cs, halves)


@pytest.mark.parametrize("halves", [False, True])
def test_rope_of_slices_in_place(halves):
    """q and k as column slices of one projection, turned in place; v and the rows around stay as they were."""
    L, H, D = 45, 3, 128
    z = rand((L + 2, 3 * H * D), 5).cuda()
    old = z.clone()
    cs = tern.rope_table(torch.arange(L).float()[:, None].cuda(), (128,))
    q = z[1:L + 1, :H * D].view(L, H, D)
    k = z[1:L + 1, H * D:2 * H * D].view(L, H, D)
    got = tern.rope([q, k], cs, halves=halves, outs=[q, k])
    assert got[0].data_ptr() == q.data_ptr()
    turned_close(q, old[1:L + 1, :H * D].view(L, H, D), cs, halves)
    turned_close(k, old[1:L + 1, H * D:2 * H * D].view(L, H, D), cs, halves)
    assert torch.equal(z[:, 2 * H * D:], old[:, 2 * H * D:])
    assert torch.equal(z[0], old[0]) and torch.equal(z[-1], old[-1])


@pytest.mark.parametrize("per_batch", [False, True])
def test_rope_of_a_batch(per_batch):
    """[B, L, H, D] against a table shared by the batch or one row per entry and token; one input heads-first."""
    B, L, H, D = 3, 21, 4, 64
    n = B * L if per_batch else L
    ids = torch.arange(n).float()[:, None].cuda() * 3
    cs = tern.rope_table(ids, (64,))
    x0 = rand((B, L, H, D), 1).cuda()
    x1 = rand((B, H, L, D), 2).cuda().transpose(1, 2)
    y0, y1 = tern.rope([x0, x1], cs)
    c = cs.view(B, L, 32, 2) if per_batch else cs[None].expand(B, L, 32, 2)
    turned_close(y0, x0, c, False)
    turned_close(y1, x1, c, False)
    out = torch.empty(B, H, L, D, dtype=torch.bfloat16, device="cuda").transpose(1, 2)  # heads-first output
    tern.rope([x0], cs, outs=[out])
    assert torch.equal(out, y0)


def test_rope_of_a_broadcast_input_and_of_nothing():
    L, H, D = 9, 5, 32
    cs = tern.rope_table(torch.arange(L).float()[:, None].cuda(), (32,))
    x = rand((L, 1, D), 4).cuda().expand(L, H, D)
    y, = tern.rope([x], cs)
    turned_close(y, x, cs, False)
    assert tern.rope([], cs) == []
    e, = tern.rope([rand((0, H, D), 1).cuda()], cs[:0].contiguous())
    assert e.shape == (0, H, D)


def test_rope_behind_32_bit_offsets():
    """Head rows more than 2^32 bytes apart."""
    L, D = 3, 64
    big = torch.empty(L * (1 << 31) // 2 + D, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((L, 1, D), ((1 << 31) // 2 * 1, D, 1))
    x.copy_(rand((L, 1, D), 8))
    far = torch.empty((1 << 32) + D, dtype=torch.bfloat16, device="cuda").as_strided((2, 1, D), (1 << 32, D, 1))
    far.copy_(rand((2, 1, D), 9))
    cs = tern.rope_table(torch.arange(L).float()[:, None].cuda(), (64,))
    y, = tern.rope([x], cs)
    turned_close(y, x, cs, False)
    y, = tern.rope([far], cs[:2].contiguous())
    turned_close(y, far, cs[:2], False)


def test_rope_on_another_stream_and_in_a_graph():
    L, H, D = 64, 2, 128
    ids = torch.arange(3 * L).view(L, 3).float().cuda()
    x = rand((L, H, D), 6).cuda()
    want_cs = tern.rope_table(ids, (16, 56, 56))
    want, = tern.rope([x], want_cs)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    cs = tern.rope_table(ids, (16, 56, 56), stream=s)
    y, = tern.rope([x], cs, stream=s)
    s.synchronize()
    assert torch.equal(cs, want_cs) and torch.equal(y, want)
    out, tab = torch.zeros_like(x), torch.zeros_like(cs)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tern.rope_table(ids, (16, 56, 56), out=tab)
        tern.rope([x], tab, outs=[out])
    x.copy_(rand((L, H, D), 7))
    ids.add_(5)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(tab, tern.rope_table(ids, (16, 56, 56)))
    assert torch.equal(out, tern.rope([x], tab)[0])
