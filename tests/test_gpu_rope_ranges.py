"""tern_rope and tern_rope_table at the ends of their documented ranges, on the GPU."""
from __future__ import annotations

import numpy as np
import pytest
import torch

from bit_post_quantised_b200 import tern
from oracle import block_ops as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [2 ** 31 - 1, 2 ** 31 - 64])
def test_rotation_of_as_many_rows_as_there_may_be(rows):
    """One broadcast token for each of the last row counts below 2^31 (64 GB of
    output): every row is the rotation of that token."""
    D = 16
    cs = tern.rope_table(torch.tensor([[0.75]], device="cuda"), (D,))
    x = torch.randn(1, 1, 1, D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    want = tern.rope([x], cs)[0].view(D)
    y = torch.empty(rows, 1, 1, D, dtype=torch.bfloat16, device="cuda")
    try:
        y[-1] = 0.0
        tern.rope([x.expand(rows, 1, 1, D)], cs, outs=[y])
        words = y.view(-1).view(torch.int64).view(rows, D // 4)
        ref = want.view(torch.int64)
        for at in range(0, rows, 1 << 27):
            assert (words[at:at + (1 << 27)] == ref).all()
    finally:
        del y
        words = None
        torch.cuda.empty_cache()


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("layout", ["between heads", "heads first", "entries first"])
def test_rotation_in_place_of_slices_that_lie_between_one_another(layout, halves):
    """q and k of a projection whose heads hold q, k and v side by side, or of
    a tensor [B, 3, H, L, D] or [3, B, L, H, D]: turned in place, v as it was."""
    B, L, H, D = 2, 37, 5, 64
    g = torch.Generator().manual_seed(2)
    shape, order = {"between heads": ((B, L, H, 3, D), (0, 1, 2, 3, 4)), "heads first": ((B, 3, H, L, D), (0, 3, 2, 1, 4)),
                    "entries first": ((3, B, L, H, D), (1, 2, 3, 0, 4))}[layout]
    z = torch.randn(shape, generator=g).to(torch.bfloat16).cuda().permute(order)
    q, k, v = (z[:, :, :, i] for i in range(3))
    cs = tern.rope_table(torch.arange(L).float()[:, None].cuda(), (48,))
    want = tern.rope([q.clone(), k.clone()], cs, halves=halves)
    keep = v.clone()
    tern.rope([q, k], cs, halves=halves, outs=[q, k])
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, keep)


@pytest.mark.parametrize("L,axes", [(70, (42, 42, 42)), (33, (62,)), (1, (6,)), (97, (2, 200, 48, 4))])
def test_tables_of_odd_pair_counts(L, axes):
    """One rounding to fp32 (2^-24 relative), the 64-bit angle's error (2^-50 of
    it) and the polynomials' truncation (below 1e-11), as for even counts."""
    ids = torch.randint(-50, 5000, (L, len(axes)), generator=torch.Generator().manual_seed(L)).float()
    ang, want = ref.rope_angles(ids.numpy(), axes, 1e4), ref.rope_table(ids.numpy(), axes, 1e4)
    out = torch.full((L + 1, sum(axes) // 2, 2), 7.0, device="cuda")
    got = tern.rope_table(ids.cuda(), axes, out=out[:L]).cpu().double().numpy()
    assert np.all(np.abs(got - want) <= ref.F32 * np.abs(want) + (np.abs(ang) * 2.0 ** -50)[..., None] + 1e-11)
    assert (out[L] == 7).all()
