"""The operators between the ternary linears of a conditioned image or video
transformer block, as cases to measure: rotary tables of several axes, the
rotation of queries and keys, attention to an encoder's states, and the gated
residual update with the norms around it.

``own`` selects what ``run`` calls: elementary torch operations in 32 bits
(False), or this repository's operators (True).
"""
import math

import torch

own = False

THETA = 10000.0


# ---------------------------------------------------------------------- cases
def _table(name, L, axes):
    return dict(name=name, op="table", L=L, axes=axes)


def _rope(name, L, H, Hk, D, axes, halves, fused):
    return dict(name=name, op="rope", L=L, H=H, Hk=Hk, D=D, axes=axes, halves=halves, fused=fused)


def _attn(name, B, Lq, Lk, H, Hkv, D, mask="none", fused=False):
    return dict(name=name, op="attention", B=B, Lq=Lq, Lk=Lk, H=H, Hkv=Hkv, D=D, mask=mask, fused=fused)


def _norm(name, B, T, K, post, tanh, alpha, pre, affine):
    return dict(name=name, op="norm", B=B, T=T, K=K, post=post, tanh=tanh, alpha=alpha, pre=pre, affine=affine)


def listed():
    return [
        # The small test transformer's tokens (24 of text, 8 x 8 of image): the call's latency.
        _table("table 88 tokens", 88, "16,56,56"),
        # A clip of 16 frames of 45 x 80 patches behind 77 text tokens, (time, height, width).
        _table("table clip", 16 * 45 * 80 + 77, "44,42,42"),
        # Queries and keys of one 1024 x 1024 image with its text, slices of the fused projection.
        _rope("rope image qkv", 4608, 24, 24, 128, "16,56,56", False, True),
        # A clip of 21 frames of 30 x 52 patches, half-split channel pairs.
        _rope("rope clip halves", 21 * 30 * 52, 12, 12, 128, "44,42,42", True, False),
        # One pooling query over a text encoder's 512 states.
        _attn("attention one query", 1, 1, 512, 24, 24, 128),
        # 17 latent queries of grouped heads over padded image-encoder states, lengths by request.
        _attn("attention latents", 3, 17, 1531, 16, 4, 64, "len"),
        # The 4096 image tokens of one 1024 x 1024 image over 512 text states.
        _attn("attention image to text", 1, 4096, 512, 24, 24, 128),
        # Three images of an odd size over padded text states with masked tokens inside, one prompt empty.
        _attn("attention padded batch", 3, 1021, 333, 20, 10, 96, "mask"),
        # All text and image tokens of one 1024 x 1024 image over themselves, slices of the fused projection.
        _attn("attention joint", 1, 4608, 4608, 24, 24, 128, "none", True),
        # The small test transformer's stream: the call's latency.
        _norm("norm 88 rows", 1, 88, 256, "none", False, 1.0, "layer", False),
        # One image's stream after its attention projection, before its MLP.
        _norm("norm image stream", 1, 4608, 3072, "none", False, 1.0, "layer", False),
        # Norms on both sides of the block, tanh gates of a batch of two clips, an odd width.
        _norm("norm sandwich", 2, 7021, 2312, "rms", True, 0.5, "rms", True),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def _axes(rng, rot):
    """rot channels over one to three axes, each even."""
    n = rng.choice((1, 2, 3, 3))
    cuts = sorted(rng.sample(range(1, rot // 2), n - 1))
    return ",".join(str(2 * (b - a)) for a, b in zip([0] + cuts, cuts + [rot // 2]))


def draw(rng):
    op = rng.choice(("table", "rope", "attention", "attention", "norm"))
    if op == "table":
        c = _table("", _log(rng, 1, 57000), _axes(rng, rng.choice((32, 64, 96, 128))))
    elif op == "rope":
        D = rng.choice((64, 80, 96, 128))
        H = rng.choice((1, 2, 5, 8, 12, 16, 24))
        c = _rope("", _log(rng, 1, 32000 * 12 * 128 // (max(H, 4) * D) if H > 12 else 30000), H,
                  rng.choice([h for h in (1, 2, 5, 8, 12, 16, 24) if h <= H]), D,
                  _axes(rng, rng.choice([r for r in (32, 64, 80, 96, 128) if r <= D])), rng.random() < 0.4, rng.random() < 0.5)
    elif op == "attention":
        D = rng.choice((64, 64, 72, 80, 96, 128, 128, 128))
        Hkv, G, B = rng.choice((1, 2, 4, 8, 12, 16, 24)), rng.choice((1, 1, 1, 2, 4)), rng.choice((1, 1, 2, 3, 4))
        few = rng.random() < 0.4
        Lq = _log(rng, 1, 40) if few else _log(rng, 40, 5000)
        Lk = _log(rng, 1, 12000) if few else _log(rng, 16, 5000)
        H = min(Hkv * G, 32) // Hkv * Hkv
        top = 4.0 * 4608 * 4608 * 24 * 128
        Lq = max(1, min(Lq, int(top / (4.0 * B * H * 128 * Lk))))
        c = _attn("", B, Lq, Lk, H, Hkv, D, rng.choice(("none", "len", "mask")), B == 1 and Lq == Lk)
    else:
        B = rng.choice((1, 1, 2, 3))
        K = 8 * _log(rng, 8, 1024)
        T = _log(rng, 1, 14042 * 2312 / (B * K))
        c = _norm("", B, T, K, rng.choice(("none", "rms", "layer")), rng.random() < 0.4, rng.choice((1.0, 0.5, 1.75)),
                  rng.choice(("none", "rms", "layer")), rng.random() < 0.5)
    del c["name"]
    return c


def _lens(c):
    """The valid keys of each padded request: all of them first, then less; the third has none."""
    full = [1.0, 0.61, 0.0, 0.27]
    return [int(c["Lk"] * full[b % 4]) for b in range(c["B"])]


# --------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _ints(text):
    return [int(v) for v in text.split(",")]


def _ids(c, g):
    """Token positions [L, axes]: rows of a grid counted from a start drawn by the seed."""
    n = len(_ints(c["axes"]))
    at = torch.arange(c["L"], device="cuda")
    start = torch.randint(0, 64, (n,), generator=g, device="cuda")
    parts = [at // 3600, at // 80 % 45, at % 80] if n == 3 else [at // 80, at % 80] if n == 2 else [at]
    return (torch.stack(parts, 1) + start).float()


def prepare(case, seed):
    c, g = case, _gen(seed)
    bf = torch.bfloat16
    if c["op"] == "table":
        return {"c": c, "ids": _ids(c, g)}
    if c["op"] == "rope":
        ids, ang = _ids(c, g).double(), []
        for a, d in enumerate(_ints(c["axes"])):
            ang.append(ids[:, a:a + 1] * THETA ** (-torch.arange(0, d, 2, device="cuda").double() / d))
        ang = torch.cat(ang, 1)
        cs = torch.stack([ang.cos(), ang.sin()], -1).float()
        L, H, Hk, D = c["L"], c["H"], c["Hk"], c["D"]
        if c["fused"]:  # [q | k | v] of one projection
            z = _randn(g, L, (H + 2 * Hk) * D).to(bf)
            q, k = z[:, :H * D].view(L, H, D), z[:, H * D:(H + Hk) * D].view(L, Hk, D)
        else:
            q, k = _randn(g, L, H, D).to(bf), _randn(g, L, Hk, D).to(bf)
        return {"c": c, "cs": cs, "q": q, "k": k}
    if c["op"] == "attention":
        B, Lq, Lk, H, Hkv, D = (c[n] for n in ("B", "Lq", "Lk", "H", "Hkv", "D"))
        # Normalised heads with learned gains: logits of about two in standard deviation.
        if c["fused"]:  # [q | k | v] of one projection
            z = _randn(g, B, Lq, (H + 2 * Hkv) * D)
            z[..., :(H + Hkv) * D] *= 1.4
            z = z.to(bf)
            q, k, v = (z[..., :H * D].view(B, Lq, H, D), z[..., H * D:(H + Hkv) * D].view(B, Lk, Hkv, D),
                       z[..., (H + Hkv) * D:].view(B, Lk, Hkv, D))
        else:  # queries of one projection, [k | v] of another
            q = (_randn(g, B, Lq, H, D) * 1.4).to(bf)
            z = _randn(g, B, Lk, 2 * Hkv * D)
            z[..., :Hkv * D] *= 1.4
            z = z.to(bf)
            k, v = z[..., :Hkv * D].view(B, Lk, Hkv, D), z[..., Hkv * D:].view(B, Lk, Hkv, D)
        s = {"c": c, "q": q, "k": k, "v": v, "kv_len": None, "key_mask": None}
        if c["mask"] != "none":
            s["kv_len"] = torch.tensor(_lens(c), dtype=torch.int32, device="cuda")
        if c["mask"] == "mask":
            s["key_mask"] = torch.rand(B, Lk, generator=g, device="cuda") < 0.8
        return s
    B, T, K = c["B"], c["T"], c["K"]
    s = {"c": c, "x": (_randn(g, B * T, K) * 2).to(bf), "o": (_randn(g, B * T, K) * 1.5 + 0.2).to(bf)}
    mod = (_randn(g, B, 3 * K) * 0.3).to(bf)  # gate, shift, scale of each batch entry
    s["gate"], s["shift"], s["scale"] = mod[:, :K], mod[:, K:2 * K], mod[:, 2 * K:]
    w = (_randn(g, 2, K) * 0.1 + 1).to(bf)
    s["post_weight"] = w[0] if c["affine"] and c["post"] != "none" else None
    s["pre_weight"] = w[1] if c["affine"] and c["pre"] != "none" else None
    return s


# ----------------------------------------------------------------- plain forms
def _plain_table(s):
    ids, ang = s["ids"].double(), []
    for a, d in enumerate(_ints(s["c"]["axes"])):
        omega = THETA ** (-torch.arange(0, d, 2, dtype=torch.float64, device=ids.device) / d)
        ang.append(ids[:, a:a + 1] * omega)
    ang = torch.cat(ang, 1)
    return torch.stack([ang.cos(), ang.sin()], -1).float()


def _plain_rotate(x, cs, halves):
    R = 2 * cs.shape[1]
    f, cos, sin = x.float(), cs[:, None, :, 0], cs[:, None, :, 1]
    if halves:
        a, b = f[..., :R // 2], f[..., R // 2:R]
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    else:
        a, b = f[..., 0:R:2], f[..., 1:R:2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    return torch.cat([y, f[..., R:]], -1).to(x.dtype)


def _plain_attention(s):
    q, k, v = (s[n].float().transpose(1, 2) for n in ("q", "k", "v"))
    B, H, Lq, D = q.shape
    Hkv, Lk = k.shape[1], k.shape[2]
    valid = torch.ones(B, Lk, dtype=torch.bool, device=q.device)
    if s["kv_len"] is not None:
        valid = valid & (torch.arange(Lk, device=q.device)[None] < s["kv_len"][:, None])
    if s["key_mask"] is not None:
        valid = valid & s["key_mask"]
    q = q.reshape(B, Hkv, H // Hkv * Lq, D)
    z = torch.matmul(q, k.transpose(2, 3)) * (1 / math.sqrt(D))
    z = z.masked_fill(~valid[:, None, None, :], -math.inf)
    top = z.amax(-1, keepdim=True)
    p = torch.exp(z - top.masked_fill(top == -math.inf, 0.0))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / total.masked_fill(total == 0, 1.0)
    return o.view(B, H, Lq, D).transpose(1, 2).to(s["q"].dtype).contiguous()


def _plain_normed(f, kind, weight, eps=1e-6):
    if kind == "layer":
        f = f - f.mean(-1, keepdim=True)
    if kind != "none":
        f = f * torch.rsqrt(f.square().mean(-1, keepdim=True) + eps)
    return f if weight is None else f * weight.float()


def _plain_norm(s):
    c = s["c"]
    T = c["T"]
    gate, shift, scale = (s[n].float().repeat_interleave(T, 0) for n in ("gate", "shift", "scale"))
    gate = torch.tanh(gate) if c["tanh"] else gate
    r = c["alpha"] * s["x"].float() + gate * _plain_normed(s["o"].float(), c["post"], s["post_weight"])
    if c["pre"] == "none":
        return [r.to(s["x"].dtype)]
    h = _plain_normed(r, c["pre"], s["pre_weight"]) * (1 + scale) + shift
    return [r.to(s["x"].dtype), h.to(s["x"].dtype)]


def run(state):
    s, c = state, state["c"]
    if own:
        return _run_own(s, c)
    if c["op"] == "table":
        return _plain_table(s)
    if c["op"] == "rope":
        return [_plain_rotate(s[n], s["cs"], c["halves"]) for n in ("q", "k")]
    if c["op"] == "attention":
        return _plain_attention(s)
    return _plain_norm(s)


def _run_own(s, c):
    from bit_post_quantised_b200 import tern

    if c["op"] == "table":
        return tern.rope_table(s["ids"], _ints(c["axes"]), THETA)
    if c["op"] == "rope":
        return tern.rope([s["q"], s["k"]], s["cs"], halves=c["halves"])
    if c["op"] == "attention":
        return tern.attention(s["q"], s["k"], s["v"], kv_len=s["kv_len"], key_mask=s["key_mask"])
    kinds = {"none": tern.NORM_NONE, "rms": tern.NORM_RMS, "layer": tern.NORM_LAYER}
    x, h = tern.gated_residual_norm(
        s["x"], s["o"], gate=s["gate"], gate_tanh=c["tanh"], residual_scale=c["alpha"], post_norm=kinds[c["post"]],
        post_weight=s["post_weight"], post_eps=1e-6, pre_norm=kinds[c["pre"]], pre_weight=s["pre_weight"], pre_eps=1e-6,
        scale=s["scale"] if c["pre"] != "none" else None, shift=s["shift"] if c["pre"] != "none" else None,
        tokens_per_row=c["T"])
    return [x] if h is None else [x, h]


# ----------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "table":
        pairs = sum(_ints(c["axes"])) // 2
        return {"bytes": c["L"] * (4 * len(_ints(c["axes"])) + 8 * pairs), "flops": 40 * c["L"] * pairs}
    if c["op"] == "rope":
        heads, rot = c["H"] + c["Hk"], sum(_ints(c["axes"]))
        return {"bytes": c["L"] * (4 * heads * c["D"] + 4 * rot), "flops": 3 * c["L"] * heads * rot}
    if c["op"] == "attention":
        keys = [c["Lk"]] * c["B"] if c["mask"] == "none" else _lens(c)
        return {"bytes": 4 * c["B"] * c["Lq"] * c["H"] * c["D"] + 4 * sum(keys) * c["Hkv"] * c["D"]
                + (sum(keys) if c["mask"] == "mask" else 0),
                "flops": 4 * c["Lq"] * sum(keys) * c["H"] * c["D"] + 1}
    n = c["B"] * c["T"] * c["K"]
    return {"bytes": (6 if c["pre"] == "none" else 8) * n + 6 * c["B"] * c["K"], "flops": 16 * n}


# ---------------------------------------------------------------------- exact
def exact(case, seed):
    """The operators from their definitions in 64 bits."""
    c, s = case, prepare(case, seed)
    f64 = torch.float64
    if c["op"] == "table":
        out = torch.empty(c["L"], sum(_ints(c["axes"])) // 2, 2, dtype=f64, device="cuda")
        j0 = 0
        for a, d in enumerate(_ints(c["axes"])):
            for j in range(d // 2):
                turn = s["ids"][:, a].to(f64) / math.pow(THETA, 2 * j / d)
                out[:, j0 + j, 0], out[:, j0 + j, 1] = torch.cos(turn), torch.sin(turn)
            j0 += d // 2
        return out
    if c["op"] == "rope":
        turn = torch.view_as_complex(s["cs"].to(f64).contiguous())[:, None, :]
        n = turn.shape[-1]
        got = []
        for name in ("q", "k"):
            x = s[name].to(f64)
            pair = x[..., :2 * n].unflatten(-1, (2, n) if c["halves"] else (n, 2))
            pair = pair.transpose(-1, -2) if c["halves"] else pair
            y = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn)
            y = y.transpose(-1, -2) if c["halves"] else y
            got.append(torch.cat([y.reshape(*x.shape[:-1], 2 * n), x[..., 2 * n:]], -1))
        return got
    if c["op"] == "attention":
        o = torch.zeros(s["q"].shape, dtype=f64, device="cuda")
        for b in range(c["B"]):
            keep = torch.arange(c["Lk"], device="cuda")
            if s["kv_len"] is not None:
                keep = keep[:int(s["kv_len"][b])]
            if s["key_mask"] is not None:
                keep = keep[s["key_mask"][b, :len(keep)]]
            if not len(keep):
                continue
            for h in range(c["H"]):
                k, v = (s[n][b, keep, h // (c["H"] // c["Hkv"])].to(f64) for n in ("k", "v"))
                z = s["q"][b, :, h].to(f64) @ k.T / c["D"] ** 0.5
                z = torch.exp(z - torch.logsumexp(z, 1)[:, None])
                o[b, :, h] = z @ v
        return o
    x, o = s["x"].to(f64), s["o"].to(f64)
    K, row = c["K"], torch.arange(len(x), device="cuda") // c["T"]

    def normed(t, kind, w):
        if kind == "none":
            return t
        if kind == "layer":
            t = t - t.sum(1)[:, None] / K
        t = t / torch.sqrt((t * t).sum(1)[:, None] / K + 1e-6)
        return t * w.to(f64) if w is not None else t

    gate = s["gate"].to(f64)
    r = x * c["alpha"] + normed(o, c["post"], s["post_weight"]) * (torch.tanh(gate) if c["tanh"] else gate)[row]
    if c["pre"] == "none":
        return [r]
    return [r, normed(r, c["pre"], s["pre_weight"]) * (1 + s["scale"].to(f64)[row]) + s["shift"].to(f64)[row]]
