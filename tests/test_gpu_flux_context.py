"""The block forward with an encoder's states as context, on the GPU: the
rotary table, attention to the states, the rotation and the gated update with
its norms run together, as the model uses them, against the fp64 block oracle.

Small config and bars as the forward without context has them (rounding
decisions that flip, bf16 probabilities): |out - ref| <= 2^-5 (|ref| +
rms(ref)) and rms(out - ref) <= 2^-7 rms(ref).
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle
from oracle import flux as OF
from bit_post_quantised_b200 import flux, tern, workloads

pytestmark = pytest.mark.gpu
DIM = 192


def ternary(q, b=None):
    packed, scales, bias = q
    K = packed.numel() * 4 // (-(-scales.shape[0] // 128) * 128)
    T, bad = oracle.unpack_tiled(packed.cpu().numpy(), scales.shape[0], K)
    assert bad == 0
    return T, scales.cpu().double().numpy(), workloads.bf16_bits(bias.cpu())


@pytest.fixture(scope="module")
def small():
    cfg = workloads.FLUX_SMALL
    weights = {(k, 0): workloads.flux_block_weights(cfg, k, 0) for k in ("double", "single")}
    weights[("context", 0)] = workloads.flux_context_weights(cfg, 0, DIM)
    model = flux.TernaryFlux(cfg, weights, device="cuda")
    p = {}
    for kind in ("double", "single"):
        p[kind] = {name: ternary(model.blocks[(kind, 0)][name]) for name, _, _ in workloads.flux_block_shapes(cfg, kind)}
        p[kind].update({k: workloads.bf16_bits(v) for k, v in weights[(kind, 0)].items() if k.endswith("_norm")})
    p["double"]["ctx.kv"] = ternary(model.context[0]["kv"])
    p["double"]["ctx.norm"] = workloads.bf16_bits(weights[("context", 0)]["norm"])
    p["double"]["ctx.gate"] = workloads.bf16_bits(weights[("context", 0)]["gate"])
    return cfg, weights, model, p


def f64(t):
    return OF.from_bits(workloads.bf16_bits(t))


def check(out: torch.Tensor, ref: np.ndarray):
    a = out.double().cpu().numpy()
    rms = float(np.sqrt(np.mean(ref ** 2)))
    d = np.abs(a - ref)
    bad = d > 2.0 ** -5 * (np.abs(ref) + rms)
    assert not bad.any(), f"{int(bad.sum())} of {bad.size} outside the bar; worst {d.max() / rms:.3e} rms"
    assert np.sqrt(np.mean(d ** 2)) <= 2.0 ** -7 * rms, f"rms diff {np.sqrt(np.mean(d ** 2)) / rms:.3e}"
    assert tern.device_status() == 0


@pytest.mark.parametrize("Lc,valid", [(19, None), (40, 23), (700, 512), (3, None)])
def test_forward_with_context_matches_oracle(small, Lc, valid):
    cfg, weights, model, p = small
    img, txt, vec, ids = workloads.flux_inputs(cfg)
    ctx = torch.randn(Lc, DIM, generator=torch.Generator().manual_seed(Lc)).to(torch.bfloat16)
    padded = ctx.clone()
    if valid is not None:
        padded[valid:] = float("nan")  # padding holds anything
    n = None if valid is None else torch.tensor([valid], dtype=torch.int32, device="cuda")
    out = model.forward(img.cuda(), txt.cuda(), vec.cuda(), ids, context=padded.cuda(), context_len=n)
    ang = OF.rope_angles(ids.numpy())
    oi, ot = OF.double_block(f64(img), f64(txt), f64(vec), p["double"], ang, f64(ctx[:valid]))
    ref = OF.single_block(np.concatenate([ot, oi]), f64(vec), p["single"], ang)
    check(out, ref)
    # the states matter: the block without them is far outside the bar
    plain, _ = OF.double_block(f64(img), f64(txt), f64(vec), p["double"], ang)
    assert np.sqrt(np.mean((plain - oi) ** 2)) > 0.1 * np.sqrt(np.mean(oi ** 2))


def test_without_states_the_forward_is_the_models_without_weights_for_them(small):
    cfg, weights, model, _ = small
    img, txt, vec, ids = (t.cuda() for t in workloads.flux_inputs(cfg))
    plain = flux.TernaryFlux(cfg, {k: v for k, v in weights.items() if k[0] != "context"}, device="cuda")
    assert torch.equal(model.forward(img, txt, vec, ids), plain.forward(img, txt, vec, ids))
    with pytest.raises(ValueError, match="no weights"):
        plain.forward(img, txt, vec, ids, context=torch.zeros(4, DIM, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="context_len"):
        model.forward(img, txt, vec, ids, context_len=torch.zeros(1, dtype=torch.int32, device="cuda"))


def test_no_valid_state_adds_nothing_but_the_rounding(small):
    """A length of zero: the attention gives zeros, whose RMS norm is zero."""
    cfg, weights, model, p = small
    img, txt, vec, ids = workloads.flux_inputs(cfg)
    ctx = torch.full((20, DIM), float("nan"), dtype=torch.bfloat16, device="cuda")
    out = model.forward(img.cuda(), txt.cuda(), vec.cuda(), ids, n_single=0, context=ctx,
                        context_len=torch.zeros(1, dtype=torch.int32, device="cuda"))
    ang = OF.rope_angles(ids.numpy())
    oi, ot = OF.double_block(f64(img), f64(txt), f64(vec), p["double"], ang)
    check(out, np.concatenate([ot, oi]))


def test_on_a_stream_and_captured(small):
    cfg, weights, model, _ = small
    img, txt, vec, ids = (t.cuda() for t in workloads.flux_inputs(cfg))
    ctx = torch.randn(77, DIM, device="cuda").to(torch.bfloat16)
    n = torch.tensor([50], dtype=torch.int32, device="cuda")
    want = model.forward(img, txt, vec, ids, context=ctx, context_len=n)
    s = torch.cuda.Stream()
    on = flux.TernaryFlux(cfg, weights, device="cuda", stream=s)
    got = on.forward(img, txt, vec, ids, context=ctx, context_len=n)
    s.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = model.forward(img, txt, vec, ids, context=ctx, context_len=n)
    n.fill_(30)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, model.forward(img, txt, vec, ids, context=ctx, context_len=n))
