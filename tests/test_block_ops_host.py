"""The operators between a block's linears, on the host: the fp64 oracle
against independent forms, and every refusal of the C ABI and the binding
before anything is launched (fake pointers, never dereferenced)."""
from __future__ import annotations

import ctypes
import struct

import numpy as np
import pytest
import torch

from bit_post_quantised_b200 import _build, flux, tern
from oracle import block_ops as ref

OK, INVALID, SHAPE, MISALIGNED = 0, -1, -2, -3
F = 0x7F0000000000


@pytest.fixture(scope="module")
def L():
    _build.build()
    return tern.lib()


# ------------------------------------------------------------- oracle pins
def test_oracle_table_against_the_block_forward():
    ids = torch.randint(0, 90, (40, 3), generator=torch.Generator().manual_seed(1)).float()
    cos, sin = flux.rope_cos_sin(ids)
    got = ref.rope_table(ids.numpy(), (16, 56, 56), flux.ROPE_THETA)
    assert np.abs(got[..., 0] - cos.numpy()).max() < 1e-7 and np.abs(got[..., 1] - sin.numpy()).max() < 1e-7


def test_oracle_rotation_against_torch_and_halves_against_pairs():
    x = torch.randn(7, 2, 128, generator=torch.Generator().manual_seed(2))
    ids = torch.arange(21).view(7, 3).float()
    cos, sin = flux.rope_cos_sin(ids)
    cs = np.stack([cos.numpy(), sin.numpy()], -1).astype(np.float64)
    xb = x.to(torch.bfloat16)
    want = flux.apply_rope(xb, cos, sin).double().numpy()
    got = ref.rope(xb.double().numpy(), cs, False)
    assert np.abs(got - want).max() <= 2.0 ** -8 * np.abs(got).max()
    # the same channels, laid out as halves
    h = np.concatenate([xb.double().numpy()[..., 0::2], xb.double().numpy()[..., 1::2]], -1)
    gh = ref.rope(h, cs, True)
    assert np.array_equal(gh[..., :64], got[..., 0::2]) and np.array_equal(gh[..., 64:], got[..., 1::2])


def test_oracle_attention_against_torch():
    g = torch.Generator().manual_seed(3)
    q, k, v = (torch.randn(2, n, h, 16, generator=g, dtype=torch.float64) for n, h in ((5, 4), (9, 2), (9, 2)))
    mask = torch.rand(2, 9, generator=g) < 0.7
    o, _, _ = ref.attention(q.numpy(), k.numpy(), v.numpy(), 0.3, None, mask.numpy())
    kk, vv = (t.repeat_interleave(2, 2).transpose(1, 2) for t in (k, v))
    want = torch.nn.functional.scaled_dot_product_attention(q.transpose(1, 2), kk, vv, scale=0.3,
                                                            attn_mask=mask[:, None, None, :]).transpose(1, 2)
    assert np.abs(o - want.numpy()).max() < 1e-13


def test_oracle_norms_against_torch():
    g = torch.Generator().manual_seed(4)
    x, o = torch.randn(6, 32, generator=g, dtype=torch.float64), torch.randn(6, 32, generator=g, dtype=torch.float64)
    w, gate, sc, sh = (torch.randn(n, 32, generator=g, dtype=torch.float64) for n in (1, 2, 2, 2))
    r, h, _, _ = ref.gated_residual_norm(x.numpy(), o.numpy(), alpha=0.5, post=1, post_w=w[0].numpy(), post_eps=1e-5,
                                         gate=gate.numpy(), tanh=True, pre=2, pre_eps=1e-6, scale=sc.numpy(),
                                         shift=sh.numpy(), tokens_per_row=3)
    row = torch.arange(6) // 3
    rt = 0.5 * x + gate.tanh()[row] * torch.nn.functional.rms_norm(o, (32,), w[0], 1e-5)
    ht = torch.nn.functional.layer_norm(rt, (32,), eps=1e-6) * (1 + sc[row]) + sh[row]
    assert np.abs(r - rt.numpy()).max() < 1e-12 and np.abs(h - ht.numpy()).max() < 1e-12


# ------------------------------------------------------------ C ABI refusals
def test_rope_table_rejects(L):
    def call(ids=F, n=10, dims=(16, 56, 56), theta=1e4, cs=F + 0x100000):
        return L.tern_rope_table(ids, n, len(dims), (ctypes.c_int * max(1, len(dims)))(*dims), theta, cs, None)
    assert call(n=-1) == INVALID and call(n=1 << 31) == SHAPE
    assert call(dims=()) == SHAPE and call(dims=(2,) * 5) == SHAPE
    assert call(dims=(3,)) == SHAPE and call(dims=(0, 4)) == SHAPE and call(dims=(-2,)) == SHAPE
    assert call(dims=(200, 58)) == SHAPE and call(dims=(1 << 30,)) == SHAPE
    assert call(theta=0.0) == INVALID and call(theta=float("nan")) == INVALID and call(theta=float("inf")) == INVALID
    assert call(ids=None) == INVALID and call(cs=None) == INVALID
    assert call(ids=F + 2) == MISALIGNED and call(cs=F + 0x100004) == MISALIGNED
    assert call(cs=F + 112) == INVALID  # inside ids
    assert L.tern_rope_table(F, 1, 1, None, 1e4, F, None) == INVALID
    assert call(n=0, ids=None, cs=None) == OK


def _rope(L, tensors, B=1, n=16, D=128, cs=F + 0x900000, rows=None, P=64, layout=0, count=None):
    arr = (tern.RopeTensor * max(1, len(tensors)))(*[tern.RopeTensor(*t) for t in tensors])
    return L.tern_rope(arr, len(tensors) if count is None else count, B, n, D, cs, n if rows is None else rows, P, layout,
                       None)


def test_rope_rejects(L):
    q = (F, F + 0x100000, 2, 0, 256, 128, 0, 256, 128)
    k = (F + 0x200000, F + 0x300000, 2, 0, 256, 128, 0, 256, 128)
    sub = lambda t, **kw: tuple(kw.get(n, v) for n, v in zip(  # noqa: E731
        ("x", "y", "h", "xb", "xl", "xh", "yb", "yl", "yh"), t))
    assert _rope(L, [q, k], layout=2) == INVALID
    assert _rope(L, [q] * 5) == SHAPE and _rope(L, [q], count=-1) == INVALID
    assert _rope(L, [q, k], n=-1) == INVALID and _rope(L, [q, k], B=1 << 16, n=1 << 16) == SHAPE
    assert _rope(L, [q, k], D=100) == SHAPE and _rope(L, [q, k], D=512, P=64) == SHAPE
    assert _rope(L, [q, k], P=72) == SHAPE and _rope(L, [q, k], P=4) == SHAPE and _rope(L, [q, k], P=12) == SHAPE
    assert _rope(L, [sub(q, h=-1)]) == INVALID and _rope(L, [sub(q, h=1 << 21)]) == SHAPE
    assert _rope(L, [q], cs=None) == INVALID and _rope(L, [q], cs=F + 0x900008) == MISALIGNED
    assert _rope(L, [q], rows=15) == INVALID
    assert _rope(L, [sub(q, x=0)]) == INVALID and _rope(L, [sub(q, y=0)]) == INVALID
    assert _rope(L, [sub(q, x=F + 8)]) == MISALIGNED and _rope(L, [sub(q, y=F + 0x100008)]) == MISALIGNED
    assert _rope(L, [sub(q, xl=260)]) == INVALID and _rope(L, [sub(q, xl=-256)]) == INVALID
    assert _rope(L, [sub(q, yl=0)]) == INVALID      # the tokens of y on top of one another
    assert _rope(L, [sub(q, yl=128)]) == INVALID    # heads into the next token
    assert _rope(L, [sub(q, yh=64)]) == INVALID     # heads into one another
    assert _rope(L, [sub(q, y=F + 256)]) == INVALID     # y over x, not in place
    assert _rope(L, [sub(q, y=F, yl=512)]) == INVALID   # the same start, other strides
    assert _rope(L, [q, sub(k, y=F + 0x100000)]) == INVALID  # two outputs
    assert _rope(L, [q, sub(k, x=F + 0x100000)]) == INVALID  # one's output is the other's input
    assert _rope(L, [q], cs=F + 0x100000) == INVALID    # the table inside y
    # equal row strides, columns that meet by one group
    a = (F, F, 2, 0, 768, 128, 0, 768, 128)
    assert _rope(L, [a, (F + 496, F + 496, 2, 0, 768, 128, 0, 768, 128)]) == INVALID
    assert _rope(L, [], B=0) == OK and _rope(L, [q], n=0) == OK and _rope(L, [sub(q, h=0)]) == OK
    if not torch.cuda.is_available():  # passes every check, up to the device query
        assert _rope(L, [a, (F + 512, F + 512, 2, 0, 768, 128, 0, 768, 128)]) in (-4, -6)


def _attn(L, **kw):
    d = dict(q=F, k=F + 0x1000000, v=F + 0x2000000, o=F + 0x3000000, B=2, Lq=16, Lk=32, H=4, Hkv=2, D=64, q_b=16 * 256,
             q_l=256, q_h=64, k_b=32 * 128, k_l=128, k_h=64, v_b=32 * 128, v_l=128, v_h=64, o_b=16 * 256, o_l=256, o_h=64,
             scale=0.125, kv_len=None, key_mask=None, mask_ld=32)
    d.update(kw)
    return L.tern_attention(ctypes.byref(tern.AttentionArgs(*[d[n] for n, _ in tern.AttentionArgs._fields_])), None)


def test_attention_rejects(L):
    assert L.tern_attention(None, None) == INVALID
    for n in ("B", "Lq", "Lk", "H", "Hkv", "D"):
        assert _attn(L, **{n: -1}) == INVALID, n
    assert _attn(L, D=68) == SHAPE and _attn(L, D=0) == SHAPE and _attn(L, D=136) == SHAPE
    assert _attn(L, Hkv=3) == SHAPE and _attn(L, Hkv=0) == SHAPE
    assert _attn(L, Lq=1 << 30) == SHAPE and _attn(L, Lk=1 << 30) == SHAPE
    assert _attn(L, B=1 << 19) == SHAPE and _attn(L, H=1 << 21, Hkv=1) == SHAPE
    for s in (0.0, -1.0, float("nan"), float("inf"), 3e38):
        assert _attn(L, scale=s) == INVALID
    for n in "qkvo":
        assert _attn(L, **{n: 0}) == INVALID and _attn(L, **{n: F + 0x5000008}) == MISALIGNED, n
    assert _attn(L, kv_len=F + 0x5000002) == MISALIGNED
    assert _attn(L, key_mask=F + 0x5000000, mask_ld=-1) == INVALID
    assert _attn(L, q_l=260) == INVALID and _attn(L, k_h=-64) == INVALID and _attn(L, v_b=12) == INVALID
    assert _attn(L, o_l=0) == INVALID and _attn(L, o_h=32) == INVALID and _attn(L, o_b=256) == INVALID
    assert _attn(L, o=F) == INVALID and _attn(L, o=F + 0x1000000 + 64) == INVALID and _attn(L, o=F + 0x2000000) == INVALID
    assert _attn(L, kv_len=F + 0x3000010) == INVALID and _attn(L, key_mask=F + 0x3000001) == INVALID
    assert _attn(L, B=0, q=0, o=0) == OK and _attn(L, Lq=0) == OK and _attn(L, H=0) == OK


def _norm(L, **kw):
    d = dict(x=F, o=F + 0x100000, x_out=F + 0x200000, h=F + 0x300000, M=16, K=256, ld_x=256, ld_o=256, ld_x_out=256,
             ld_h=256, residual_scale=1.0, post_norm=1, post_weight=None, post_eps=1e-6, gate=F + 0x400000, gate_tanh=0,
             pre_norm=2, pre_weight=None, pre_eps=1e-6, scale=F + 0x500000, shift=F + 0x600000, mod_ld=256,
             tokens_per_row=16)
    d.update(kw)
    a = tern.GatedResidualNormArgs(*[d[n] for n, _ in tern.GatedResidualNormArgs._fields_])
    return L.tern_gated_residual_norm(ctypes.byref(a), None)


def test_gated_residual_norm_rejects(L):
    assert L.tern_gated_residual_norm(None, None) == INVALID
    assert _norm(L, M=-1) == INVALID and _norm(L, K=0) == SHAPE and _norm(L, K=100) == SHAPE and _norm(L, K=16392) == SHAPE
    assert _norm(L, tokens_per_row=0) == SHAPE and _norm(L, M=1 << 31) == SHAPE
    assert _norm(L, post_norm=3) == INVALID and _norm(L, pre_norm=-1) == INVALID
    assert _norm(L, post_eps=-1.0) == INVALID and _norm(L, pre_eps=float("nan")) == INVALID
    assert _norm(L, residual_scale=float("inf")) == INVALID
    assert _norm(L, scale=None) == INVALID and _norm(L, shift=None) == INVALID
    assert _norm(L, post_norm=0, post_weight=F + 0x700000) == INVALID
    assert _norm(L, h=None) == INVALID and _norm(L, gate=None, gate_tanh=1) == INVALID
    for n in ("x", "o", "x_out"):
        assert _norm(L, **{n: None}) == INVALID
    for n in ("x", "o", "x_out", "h", "gate", "scale", "shift", "post_weight", "pre_weight"):
        assert _norm(L, **{n: F + 0x700008}) == MISALIGNED, n
    for n in ("ld_x", "ld_o", "ld_x_out", "ld_h", "mod_ld"):
        assert _norm(L, **{n: 248}) == INVALID and _norm(L, **{n: 260}) == INVALID, n
    assert _norm(L, x_out=F, ld_x_out=512) == INVALID            # x's start, other rows
    assert _norm(L, x_out=F + 512) == INVALID                    # x shifted by a row
    assert _norm(L, h=F + 0x200000) == INVALID                   # both outputs
    assert _norm(L, h=F + 0x400000) == INVALID and _norm(L, x_out=F + 0x500000) == INVALID  # a modulation row
    assert _norm(L, post_weight=F + 0x200100) == INVALID
    assert _norm(L, M=0, x=None, o=None, x_out=None) == OK


def test_packed_layouts_are_the_structures():
    """The binding packs two argument blocks without ctypes: byte for byte the ctypes mirrors of the header's."""
    v = list(range(1, 23)) + [0.5, 24, 25, 26]
    assert tern._ATTENTION.pack(*v) == bytes(tern.AttentionArgs(*v))
    v = list(range(1, 11)) + [0.5, 12, 13, 1.5, 15, 16, 17, 18, 2.5, 20, 21, 22, 23]
    assert tern._RESIDUAL_NORM.pack(*v) == bytes(tern.GatedResidualNormArgs(*v))
    v = list(range(1, 10))
    assert struct.pack("2P7q", *v) == bytes(tern.RopeTensor(*v))


# ------------------------------------------------------------ binding refusals
def bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def test_binding_refuses_what_does_not_fit():
    with pytest.raises(ValueError, match="ids"):
        tern.rope_table(torch.zeros(4, 2), (16, 16, 16))
    with pytest.raises(ValueError, match="ids"):
        tern.rope_table(torch.zeros(4, 3, dtype=torch.float64), (16, 16, 16))
    cs = torch.zeros(4, 16, 2)
    with pytest.raises(ValueError, match="bf16"):
        tern.rope([torch.zeros(4, 2, 32)], cs)
    with pytest.raises(ValueError, match="adjacent"):
        tern.rope([bf(4, 2, 64)[..., ::2]], cs)
    with pytest.raises(ValueError, match="share"):
        tern.rope([bf(4, 2, 32), bf(5, 2, 32)], cs)
    with pytest.raises(ValueError, match="cs"):
        tern.rope([bf(4, 2, 32)], cs.double())
    q, k = bf(2, 3, 4, 64), bf(2, 5, 2, 64)
    with pytest.raises(ValueError, match="batch"):
        tern.attention(q, k[0], k[0])
    with pytest.raises(ValueError, match="fit"):
        tern.attention(q, k, bf(2, 6, 2, 64))
    with pytest.raises(ValueError, match="fit"):
        tern.attention(q, k[:1], k[:1])
    with pytest.raises(ValueError, match="kv_len"):
        tern.attention(q, k, k, kv_len=torch.zeros(2, dtype=torch.int64))
    with pytest.raises(ValueError, match="key_mask"):
        tern.attention(q, k, k, key_mask=torch.ones(2, 5))
    with pytest.raises(ValueError, match="key_mask"):
        tern.attention(q, k, k, key_mask=torch.ones(2, 4, dtype=torch.bool))
    with pytest.raises(ValueError, match="key_mask"):
        tern.attention(q, k, k, key_mask=torch.ones(2, 10, dtype=torch.bool)[:, ::2])
    x = bf(6, 64)
    with pytest.raises(ValueError, match="shape"):
        tern.gated_residual_norm(x, bf(6, 72))
    with pytest.raises(ValueError, match="modulation rows"):
        tern.gated_residual_norm(x, x, gate=bf(2, 64), tokens_per_row=2)
    with pytest.raises(ValueError, match="modulation rows"):
        tern.gated_residual_norm(x, x, gate=bf(1, 56))
    with pytest.raises(ValueError, match="distance"):
        tern.gated_residual_norm(x, x, gate=bf(2, 64), scale=bf(2, 128)[:, :64], shift=bf(2, 64), tokens_per_row=3)
    with pytest.raises(ValueError, match="post_weight"):
        tern.gated_residual_norm(x, x, post_norm=1, post_weight=bf(32))


@pytest.mark.parametrize("call", [
    lambda: tern.rope_table(torch.zeros(4, 1), (32,)),
    lambda: tern.rope([bf(4, 2, 32)], torch.zeros(4, 16, 2)),
    lambda: tern.attention(bf(2, 3, 4, 64), bf(2, 5, 2, 64), bf(2, 5, 2, 64)),
    lambda: tern.gated_residual_norm(bf(6, 64), bf(6, 64)),
])
def test_binding_refuses_tensors_that_are_not_on_the_current_gpu(call):
    with pytest.raises(ValueError, match="current CUDA device"):
        call()


# -------------------------------------------------- which kernel attention takes
def test_attention_plan_refuses_and_answers_without_a_gpu(L):
    def plan(sms=148, **kw):
        d = dict(B=2, Lq=16, Lk=32, H=4, Hkv=2, D=64, q_l=256, k_l=128, v_l=128)
        d.update(kw)
        a = tern.AttentionArgs(**d)
        kernel, ctas = ctypes.c_int(-7), ctypes.c_int(-7)
        s = L.tern_attention_plan(ctypes.byref(a), sms, ctypes.byref(kernel), ctypes.byref(ctas))
        return (kernel.value, ctas.value) if s == OK else s
    n = ctypes.c_int()
    assert L.tern_attention_plan(None, 148, ctypes.byref(n), ctypes.byref(n)) == INVALID
    assert L.tern_attention_plan(ctypes.byref(tern.AttentionArgs()), 148, None, ctypes.byref(n)) == INVALID
    assert plan(Lq=-1) == INVALID and plan(D=68) == SHAPE and plan(Hkv=3) == SHAPE and plan(Lk=1 << 30) == SHAPE
    for empty in ("B", "Lq", "H"):
        assert plan(**{empty: 0}) == (tern.ATTENTION_NONE, 0)
    assert plan(Lk=0)[0] == tern.ATTENTION_ROWS
    big = dict(B=1, Lq=4096, Lk=512, H=24, Hkv=24, D=128)
    assert plan(**big) == (tern.ATTENTION_TILES, 1)
    assert plan(**big, k_l=0)[0] == tern.ATTENTION_ROWS and plan(**big, q_l=0)[0] == tern.ATTENTION_ROWS
    assert plan(B=1, Lq=256, Lk=16384, H=8, Hkv=8, D=128) == (tern.ATTENTION_TILES, 8)
    assert plan(B=1, Lq=1, Lk=512, H=24, Hkv=24, D=128)[0] == tern.ATTENTION_ROWS
    q, k = torch.empty(1, 256, 8, 128, device="meta"), torch.empty(1, 16384, 8, 128, device="meta")
    assert tern.attention_plan(q, k, k, sms=148) == tern.attention_plan(q[0], k[0], k[0], sms=148) == (tern.ATTENTION_TILES, 8)


def test_a_lost_remainder_of_the_probabilities_shows():
    """The bar that the row kernel is held to: fp64 attention whose
    probabilities are rounded to bf16 once is outside it."""
    g = torch.Generator().manual_seed(5)
    q, k, v = ((torch.randn(1, n, 4, 64, generator=g) * s).to(torch.bfloat16).double() for n, s in ((1, 1.4), (17, 1.4), (17, 1.0)))
    want, av, big = ref.attention(q.numpy(), k.numpy(), v.numpy(), 0.125)
    z = torch.einsum("bqhd,bkhd->bhqk", q, k) * 0.125
    p = torch.exp(z - z.amax(-1, keepdim=True))
    total = p.sum(-1, keepdim=True)
    for step, inside in ((ref.BF16 ** 2, False), (ref.BF16, True)):
        o = torch.einsum("bhqk,bkhd->bqhd", p.to(torch.bfloat16).double() / total, v).to(torch.bfloat16).double().numpy()
        e = ref.attention_bound(q.numpy(), k.numpy(), av, big, step)
        assert bool((np.abs(o - want) <= ref.BF16 * (np.abs(want) + e) + e).all()) == inside


def test_attention_takes_as_many_query_rows_as_documented(L):
    """B * H * Lq up to 2^34, whichever kernel they take."""
    far = dict(k=F - 0x40000000, v=F - 0x20000000, B=1, H=8, Hkv=8, D=8, q_l=8, q_h=0, k_l=64, k_h=8, v_l=64, v_h=8, o_l=64, o_h=8,
               o=F + (1 << 40))
    if not torch.cuda.is_available():  # passes every check, up to the device query
        assert _attn(L, **far, Lq=(1 << 28) + 5, Lk=3) in (-4, -6)
    assert _attn(L, **far, Lq=(1 << 30) - 1, Lk=0, kv_len=1) == MISALIGNED  # refused for that alone
    far.update(H=32, Hkv=32, o_l=256)
    assert _attn(L, **far, Lq=1 << 29, Lk=3) == SHAPE


def _heads(t):
    """(address, strides) of a [B, L, H, D] view of a bf16 tensor on the host, as if it lay at F."""
    return F + 2 * t.storage_offset(), t.stride()[:3]


def test_slices_of_one_parent_may_lie_between_one_another(L):
    """Every pair of slices of a small parent, in several layouts, against the sets of their elements."""
    if torch.cuda.is_available():
        pytest.skip("accepted calls would launch")
    B, n, H, D = 2, 3, 2, 16
    cs = dict(B=B, n=n, D=D, P=8, cs=F - 0x10000)
    parents = {"between heads": bf(B, n, H, 3, D), "heads first": bf(B, 3, H, n, D).permute(0, 3, 2, 1, 4),
               "entries first": bf(3, B, n, H, D).permute(1, 2, 3, 0, 4), "tokens last": bf(3, H, B, n, D).permute(2, 3, 1, 0, 4)}
    count = 0
    for z in parents.values():
        at = torch.arange(z.numel()).view(-1).as_strided(z.shape, z.stride())
        views = [z[:, :, :, i] for i in range(3)]
        ids = [at[:, :, :, i] for i in range(3)]
        for i in range(3):
            for off in (0, 8, 16, 24, 40, z.stride(2), z.stride(1) - 8, z.stride(0) + 8):
                for j in range(3):
                    (a, sa), (b, sb) = _heads(views[i]), _heads(views[j])
                    b += 2 * off
                    meet = bool(np.intersect1d(ids[i].numpy(), ids[j].numpy() + off).size)
                    got = _rope(L, [(a, a, H, *sa, *sa), (b, b, H, *sb, *sb)], **cs)
                    assert (got == INVALID) == meet and got in (INVALID, -4, -6), (i, j, off, got, meet)
                    count += not meet
    assert count > 50
    # attention's output between its inputs, and over one of them
    z = bf(B, n, H, 4, D)
    kw = {}
    for i, name in enumerate("qkvo"):
        a, s = _heads(z[:, :, :, i])
        kw.update({name: a, **{f"{name}_{x}": v for x, v in zip("blh", s)}})
    kw.update(B=B, Lq=n, Lk=n, H=H, Hkv=H, D=D)
    assert _attn(L, **kw) in (-4, -6) and _attn(L, **{**kw, "o": kw["o"] - 16}) == INVALID


def test_strides_that_reach_past_all_addresses_are_refused(L):
    """(B - 1) * stride of 2^68 elements: no overlap check in 64 bits holds there."""
    far = 1 << 38
    assert _rope(L, [(F, F, 1, far, 16, 16, far, 16, 16)], B=1 << 30, n=1, D=16, P=8) == INVALID
    assert _rope(L, [(F, F, 1, 16, far, 16, 16, far, 16)], B=1, n=1 << 30, D=16, P=8) == INVALID
    assert _attn(L, B=1, Lq=1 << 29, H=1, Hkv=1, q_l=far, o=F + 0x5000000) == INVALID
    assert _attn(L, B=1, Lk=1 << 29, H=1, Hkv=1, k_l=far) == INVALID and _attn(L, B=1, Lk=1 << 29, H=1, Hkv=1, v_l=far) == INVALID
    for n in ("ld_x", "ld_o", "ld_x_out", "ld_h"):
        assert _norm(L, M=(1 << 31) - 1, x=F, x_out=F, o=F + (1 << 40), h=F + (1 << 40), tokens_per_row=1 << 31,
                     **{"ld_x": 256, "ld_o": 256, "ld_x_out": 256, "ld_h": 256, n: far}) == INVALID
