"""tern_gated_residual_norm against the fp64 oracle on the GPU: one rounding to
bf16 (2^-8 relative) over the fp32 bound that the oracle derives."""
from __future__ import annotations

import itertools

import numpy as np
import pytest
import torch

from bit_post_quantised_b200 import tern
from oracle import block_ops as ref

pytestmark = pytest.mark.gpu


def rand(shape, seed, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std + mean).to(torch.bfloat16)


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def check(x, o, xo, h, **kw):
    names = dict(residual_scale="alpha", post_norm="post", post_weight="post_w", gate_tanh="tanh", pre_norm="pre",
                 pre_weight="pre_w")
    args = {names.get(k, k): (f64(v) if isinstance(v, torch.Tensor) else v) for k, v in kw.items()}
    for n in ("gate", "scale", "shift"):
        if args.get(n) is not None and args[n].ndim == 1:
            args[n] = args[n][None]
    r, hr, r_err, h_err = ref.gated_residual_norm(f64(x), f64(o), **args)
    assert np.all(np.abs(f64(xo) - r) <= ref.BF16 * (np.abs(r) + r_err) + r_err)
    if h is not None:
        assert np.all(np.abs(f64(h) - hr) <= ref.BF16 * (np.abs(hr) + h_err) + h_err)


@pytest.mark.parametrize("post,pre", list(itertools.product((0, 1, 2), (0, 1, 2))))
@pytest.mark.parametrize("M,K,T", [(1, 8, 1), (37, 256, 37), (13, 520, 5), (9, 776, 9), (64, 2312, 32), (5, 4104, 2)])
def test_matches_oracle(M, K, T, post, pre):
    G = -(-M // T)
    s = M * 31 + K
    x, o = rand((M, K), s, 2.0, 0.3).cuda(), rand((M, K), s + 1, 1.5, -0.2).cuda()
    kw = dict(gate=rand((G, K), s + 2, 0.5).cuda(), scale=rand((G, K), s + 3, 0.2).cuda(),
              shift=rand((G, K), s + 4, 0.5).cuda(), tokens_per_row=T, post_norm=post, pre_norm=pre, post_eps=1e-6,
              pre_eps=1e-5, residual_scale=0.75, gate_tanh=(K % 16 == 0))
    if post:
        kw["post_weight"] = rand((K,), s + 5, 0.1, 1.0).cuda()
    if pre:
        kw["pre_weight"] = rand((K,), s + 6, 0.1, 1.0).cuda()
    xo, h = tern.gated_residual_norm(x, o, **kw)
    check(x, o, xo, h, **kw)


@pytest.mark.parametrize("M,K", [(2, 16384), (3, 8192), (1, 3072), (300, 3072), (1000, 64), (8, 16376)])
def test_sizes_without_options(M, K):
    """The update alone, then with a layer norm; no gate, weights or modulation."""
    x, o = rand((M, K), M + K, 1.0).cuda(), rand((M, K), M + K + 1, 1.0).cuda()
    xo, h = tern.gated_residual_norm(x, o)
    assert h is None
    check(x, o, xo, None)
    xo, h = tern.gated_residual_norm(x, o, pre_norm=tern.NORM_LAYER)
    check(x, o, xo, h, pre_norm=2, pre_eps=1e-6)


def test_rows_of_modulation_output_and_strides():
    """gate, shift and scale as slices of a [B, 6K] modulation output; x and o
    column slices of wider tensors; outputs slices too, what lies around them
    as it was."""
    B, T, K = 3, 17, 264
    M = B * T
    wide = rand((M, 3 * K), 1).cuda()
    x, o = wide[:, :K], wide[:, 2 * K:]
    mod = rand((B, 6 * K), 2, 0.3).cuda()
    out = torch.full((M + 1, 2 * K + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    kw = dict(gate=mod[:, 2 * K:3 * K], shift=mod[:, 3 * K:4 * K], scale=mod[:, 4 * K:5 * K], tokens_per_row=T,
              pre_norm=tern.NORM_LAYER, post_norm=tern.NORM_RMS)
    xo, h = tern.gated_residual_norm(x, o, x_out=out[:M, :K], h=out[:M, K:2 * K], **kw)
    assert xo.data_ptr() == out.data_ptr()
    check(x, o, xo, h, pre_eps=1e-6, post_eps=1e-6, **kw)
    assert (out[:, 2 * K:] == 7).all() and (out[M] == 7).all()


@pytest.mark.parametrize("swap", [False, True])
@pytest.mark.parametrize("K", [256, 1160])
def test_in_place(K, swap):
    """x_out = x with h = o, and the reverse."""
    M = 21
    x, o = rand((M, K), 3, 2.0).cuda(), rand((M, K), 4, 1.0).cuda()
    kw = dict(gate=rand((K,), 5).cuda(), post_norm=tern.NORM_LAYER, pre_norm=tern.NORM_RMS)
    want = tern.gated_residual_norm(x, o, **kw)
    a, b = x.clone(), o.clone()
    got = tern.gated_residual_norm(a, b, x_out=b if swap else a, h=a if swap else b, **kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_constant_and_zero_rows():
    """A layer norm of a constant row is its shift; an RMS norm of a zero row is zero."""
    M, K = 4, 512
    x = torch.full((M, K), 3.0, dtype=torch.bfloat16, device="cuda")
    o = torch.zeros(M, K, dtype=torch.bfloat16, device="cuda")
    sh = rand((K,), 1).cuda()
    xo, h = tern.gated_residual_norm(x, o, post_norm=tern.NORM_RMS, pre_norm=tern.NORM_LAYER, scale=torch.zeros_like(sh),
                                     shift=sh)
    assert torch.equal(xo, x) and torch.equal(h, sh.expand(M, K))


def test_rows_that_are_not_finite_stay_in_their_rows():
    M, K = 5, 1024
    x, o = rand((M, K), 1).cuda(), rand((M, K), 2).cuda()
    want = tern.gated_residual_norm(x, o, post_norm=1, pre_norm=2)
    bad = o.clone()
    bad[2, 7], bad[3, 9] = float("nan"), float("inf")
    got = tern.gated_residual_norm(x, bad, post_norm=1, pre_norm=2)
    for i in (0, 1, 4):
        assert torch.equal(got[0][i], want[0][i]) and torch.equal(got[1][i], want[1][i])
    assert torch.isnan(got[1][2]).all() and torch.isnan(got[1][3]).all()


def test_large_mean_keeps_its_digits():
    """Rows far from zero: the variance is taken about the mean."""
    M, K = 6, 2048
    x, o = rand((M, K), 1, 0.5, 300.0).cuda(), rand((M, K), 2, 0.5, -200.0).cuda()
    xo, h = tern.gated_residual_norm(x, o, post_norm=tern.NORM_LAYER, pre_norm=tern.NORM_LAYER)
    check(x, o, xo, h, post_norm=2, pre_norm=2, post_eps=1e-6, pre_eps=1e-6)


def test_no_rows_another_stream_and_a_graph():
    K = 320
    e = torch.empty(0, K, dtype=torch.bfloat16, device="cuda")
    xo, h = tern.gated_residual_norm(e, e, pre_norm=1)
    assert xo.shape == (0, K) and h.shape == (0, K)
    x, o = rand((33, K), 1).cuda(), rand((33, K), 2).cuda()
    want = tern.gated_residual_norm(x, o, pre_norm=1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = tern.gated_residual_norm(x, o, pre_norm=1, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    a, b = torch.empty_like(x), torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tern.gated_residual_norm(x, o, pre_norm=1, x_out=a, h=b)
    o.copy_(rand((33, K), 3))
    g.replay()
    torch.cuda.synchronize()
    want = tern.gated_residual_norm(x, o, pre_norm=1)
    assert torch.equal(a, want[0]) and torch.equal(b, want[1])


@pytest.mark.parametrize("M,K,T", [(9001, 1032, 3000), (5003, 2312, 5003), (120007, 64, 999), (40010, 520, 40010)])
def test_long_walks_give_each_row_what_a_short_call_gives(M, K, T):
    """Many rows per CTA, strided and in place, against calls on a few hundred rows each."""
    wide = rand((M, 2 * K), 1).cuda()
    x, o = wide[:, :K], rand((M, K), 2).cuda()
    G = -(-M // T)
    gate, scale, shift = (rand((G, K), 3 + i, 0.5).cuda() for i in range(3))
    kw = dict(post_norm=tern.NORM_RMS, pre_norm=tern.NORM_LAYER)
    keep = wide[:, K:].clone()
    want = [torch.empty(M, K, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for m in range(0, M, 333):
        for g in range(m // T, -(-min(m + 333, M) // T)):
            a, b = max(m, g * T), min(m + 333, M, (g + 1) * T)
            tern.gated_residual_norm(x[a:b], o[a:b], gate=gate[g], scale=scale[g], shift=shift[g], x_out=want[0][a:b],
                                     h=want[1][a:b], **kw)
    got = tern.gated_residual_norm(x, o, gate=gate, scale=scale, shift=shift, tokens_per_row=T, x_out=x, h=o, **kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(wide[:, K:], keep)
