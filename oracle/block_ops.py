"""fp64 CPU forms of the operators between a block's linears (rotary table and
rotation, attention with masked keys, gated residual update with its norms),
written from their definitions in include/tern.h.  Test infrastructure only.

Every function takes numpy arrays holding the exact values of the bf16 or
fp32 inputs and returns fp64.  The ``*_bound`` results say how far a kernel
with fp32 arithmetic may be before its last rounding.
"""
from __future__ import annotations

import numpy as np

BF16 = 2.0 ** -8   # half a step of bf16, relative
F32 = 2.0 ** -24   # half a step of fp32, relative


def rope_angles(ids, axes, theta):
    """[L, P] angles: axis a's pairs turn by ids[:, a] * theta^(-2 i / d_a)."""
    cols = []
    for a, d in enumerate(axes):
        for i in range(d // 2):
            cols.append(ids[:, a].astype(np.float64) * float(theta) ** (-2.0 * i / d))
    return np.stack(cols, axis=1)


def rope_table(ids, axes, theta):
    ang = rope_angles(ids, axes, theta)
    return np.stack([np.cos(ang), np.sin(ang)], axis=-1)


def rope(x, cs, halves):
    """x [..., L, H, D] turned by cs [..., L, P, 2] (leading dimensions broadcast)."""
    P = cs.shape[-2]
    z = cs[..., 0] + 1j * cs[..., 1]
    z = z[..., None, :]
    y = np.array(x, dtype=np.float64)
    if halves:
        w = (x[..., :P] + 1j * x[..., P:2 * P]) * z
        y[..., :P], y[..., P:2 * P] = w.real, w.imag
    else:
        w = (x[..., 0:2 * P:2] + 1j * x[..., 1:2 * P:2]) * z
        y[..., 0:2 * P:2], y[..., 1:2 * P:2] = w.real, w.imag
    return y


def attention(q, k, v, scale, kv_len=None, key_mask=None):
    """softmax(scale q k^T) v over the valid keys of q [B, Lq, H, D], k, v [B,
    Lk, Hkv, D]; zeros without one.  Returns (o, sum_j p_j |v_j|, s) with s
    [B, H] the largest scale * sum_d |q_d k_jd| of a valid key."""
    B, Lq, H, D = q.shape
    G = H // k.shape[2] if k.shape[2] else 1
    o, av, big = np.zeros(q.shape), np.zeros(q.shape), np.zeros((B, H))
    for b in range(B):
        keep = np.arange(k.shape[1])
        if kv_len is not None:
            keep = keep[keep < kv_len[b]]
        if key_mask is not None:
            keep = keep[key_mask[b][keep] != 0]
        if len(keep) == 0:
            continue
        for h in range(H):
            kk, vv, qq = k[b, keep, h // G], v[b, keep, h // G], q[b, :, h]
            s = scale * (qq @ kk.T)
            p = np.exp(s - s.max(axis=1, keepdims=True))
            p /= p.sum(axis=1, keepdims=True)
            o[b, :, h], av[b, :, h] = p @ vv, p @ np.abs(vv)
            big[b, h] = scale * (np.abs(qq) @ np.abs(kk).T).max()
    return o, av, big


def attention_bound(q, k, av, big, p_step):
    """How far before its last rounding an fp32 attention may be: a score is
    off by at most (D + 3) half steps of the sum of its products' magnitudes
    (and of the subtracted maximum), which is the relative error of its
    probability, once in the sum of products and once in the denominator;
    sums over Lk keys in any order add at most Lk / 4 half steps here (the
    kernels' chains are that short), the exponential 2^-20; `p_step` is the
    relative half step at which probabilities enter the second product."""
    D, Lk = q.shape[-1], k.shape[1]
    score = (2 * D + 8) * F32 * big[:, None, :, None]
    return av * (2 * score + (Lk / 4 + 16) * F32 + 2.0 ** -20 + p_step)


def _normed(v, kind, eps, w):
    if kind == 2:
        v = v - v.mean(axis=1, keepdims=True)
    rstd = np.ones((v.shape[0], 1))
    if kind:
        rstd = 1.0 / np.sqrt((v * v).mean(axis=1, keepdims=True) + eps)
    v = v * rstd
    return (v if w is None else v * w), rstd


def gated_residual_norm(x, o, alpha=1.0, post=0, post_w=None, post_eps=0.0, gate=None, tanh=False, pre=0, pre_w=None,
                        pre_eps=0.0, scale=None, shift=None, tokens_per_row=None):
    """(r, h) and how far an fp32 evaluation of each may be before its last
    rounding.  Statistics over K values in fp32 are within 64 half steps of
    the mean magnitude (chains of at most 64 additions); a normalised value
    also carries its own subtraction's."""
    M = x.shape[0]
    row = np.arange(M) // (tokens_per_row or max(M, 1))
    n, rstd = _normed(o, post, post_eps, post_w)
    mag = np.abs(o) + (np.abs(o).mean(axis=1, keepdims=True) if post == 2 else 0)
    n_err = (64 * F32 * (np.abs(n) + mag * rstd * (1 if post_w is None else np.abs(post_w)))) if post else 0 * o
    g = np.ones((1, x.shape[1]))[np.zeros(M, int)] if gate is None else (np.tanh(gate) if tanh else gate)[row]
    r = alpha * x + g * n
    r_err = np.abs(g) * n_err + 8 * F32 * (np.abs(alpha * x) + np.abs(g * n))
    h, rstd = _normed(r, pre, pre_eps, pre_w)
    wmag = 1 if pre_w is None else np.abs(pre_w)
    mag = np.abs(r) + (np.abs(r).mean(axis=1, keepdims=True) if pre == 2 else 0)
    if pre:
        # r's own error reaches h directly and, at most by its root mean
        # square relative to the row's, through the statistics
        through = np.sqrt((r_err ** 2).mean(axis=1, keepdims=True)) * rstd
        h_err = r_err * rstd * wmag + 2 * through * (wmag + np.abs(h)) + 64 * F32 * (np.abs(h) + mag * rstd * wmag)
    else:
        h_err = r_err
    if scale is not None:
        h_err = h_err * np.abs(1 + scale[row]) + 4 * F32 * (np.abs(h * (1 + scale[row])) + np.abs(shift[row]))
        h = h * (1 + scale[row]) + shift[row]
    return r, h, r_err, h_err
