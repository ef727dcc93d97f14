"""What is measured of the operators around the hybrid attention in a video-DiT block.

Two operators, each with its gradient:

  residual_norm   x_out = rs * x + gate * post(y);  h = norm(x_out) * (1 + scale) + shift
                  the end of one block (gated residual, optionally with an RMS norm of the block's
                  output) and the start of the next one (modulated norm), in one pass.  The modulation
                  vectors are per sample, per latent frame or per token.
  qk_rope         q, k = rotate(rms_norm(q) * wq), rotate(rms_norm(k) * wk)
                  QK norm (none, per head or over all heads of a token) and the rotary positions of the
                  (t, h, w) axes.

A case says which operator, which direction and at which sizes and types; `run` computes it in plain
torch operations, or with the framework's calls where `own` is set.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------------------------------- cases
def _norm_case(name, direction, batch, tokens, channels, groups, norm, post, stream, block, mod, weights, residual,
               residual_scale=1.0):
    """groups: modulation rows per sample; weights: type of the norms' weights, or "none"; residual: whether
    there is a block output y to add (else the operator is the norm before the first block)."""
    return {"name": name, "op": "residual_norm", "direction": direction, "batch": batch, "tokens": tokens,
            "channels": channels, "groups": groups, "norm": norm, "post": post, "stream": stream, "block": block,
            "mod": mod, "weights": weights, "residual": residual, "residual_scale": residual_scale}


def _rope_case(name, direction, batch, T, H, W, tokens, first, heads, kv_heads, head_dim, norm, x, out, weights,
               positions="grid", pairing="interleaved", schedule="axis", fused=False, theta=1e4):
    """tokens from `first` on of the T x H x W grid (positions "grid"), or tokens at listed positions."""
    return {"name": name, "op": "qk_rope", "direction": direction, "batch": batch, "T": T, "H": H, "W": W,
            "tokens": tokens, "first": first, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim,
            "norm": norm, "x": x, "out": out, "weights": weights, "positions": positions, "pairing": pairing,
            "schedule": schedule, "fused": fused, "theta": theta}


def listed():
    n, r = _norm_case, _rope_case
    return [
        # a single token of a streaming generator at the small model's width: latency
        n("norm-token", "fwd", 1, 1, 1536, 1, "layer", "none", "f32", "bf16", "f32", "none", True),
        # the small video model's whole latent, residual stream kept in fp32
        n("norm-480p-f32-stream", "fwd", 1, 32760, 1536, 1, "layer", "none", "f32", "bf16", "f32", "none", True),
        # the large video model's latent at 720p
        n("norm-720p", "fwd", 1, 75600, 5120, 1, "layer", "none", "bf16", "bf16", "f32", "none", True),
        # a sandwich of RMS norms with weights, ragged batch of image latents, fp16
        n("norm-sandwich-ragged", "fwd", 3, 1239, 2056, 7, "rms", "rms", "f16", "f16", "f16", "f16", True, 0.75),
        # training, one modulation row per latent frame, fp32 stream and affine norm
        n("norm-480p-frames-bwd", "bwd", 1, 32760, 1536, 21, "layer", "none", "f32", "bf16", "f32", "f32", True),
        # training at the large model's size
        n("norm-720p-bwd", "bwd", 1, 75600, 5120, 1, "layer", "none", "bf16", "bf16", "f32", "none", True),
        # one new token per request: QK norm over all heads, rotation far into the grid
        r("rope-token", "fwd", 4, 21, 30, 52, 1, 30001, 12, 12, 128, "token", "bf16", "bf16", "bf16", fused=True),
        # the small model's latent out of one fused projection
        r("rope-480p-fused", "fwd", 1, 21, 30, 52, 32760, 0, 12, 12, 128, "token", "bf16", "bf16", "bf16", fused=True),
        # the large model's latent, norm per head
        r("rope-720p", "fwd", 1, 21, 45, 80, 75600, 0, 40, 40, 128, "head", "bf16", "bf16", "f32"),
        # packed images and text at listed positions, fewer key heads, halves paired, fp16
        r("rope-listed-halves", "fwd", 3, 16, 64, 64, 1021, 0, 14, 2, 64, "head", "f16", "f16", "f16",
          positions="listed", pairing="halves", schedule="shared", theta=1e6),
        # training: gradients come in fp32 as the attention's backward writes them
        r("rope-480p-bwd", "bwd", 1, 21, 30, 52, 32760, 0, 12, 12, 128, "token", "bf16", "f32", "f32"),
        r("rope-720p-bwd", "bwd", 1, 21, 45, 80, 75600, 0, 40, 40, 128, "head", "bf16", "bf16", "f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.5:
        channels = 8 * _log_int(rng, 8, 1024)
        batch = rng.choice([1, 1, 2, 3, 5])
        tokens = max(1, min(_log_int(rng, 1, 75600), 75600 * 5120 // (channels * batch) // 2))
        per = rng.choice(["sample", "frame", "token"])
        groups = 1 if per == "sample" else tokens
        if per == "frame":
            groups = min(tokens, rng.randint(2, 33))
            tokens = tokens // groups * groups
        stream, block = rng.choice([("bf16", "bf16"), ("f32", "bf16"), ("f16", "f16"), ("f32", "f16"), ("f32", "f32")])
        residual = rng.random() < 0.8
        c = _norm_case("", rng.choice(["fwd", "bwd"]), batch, tokens, channels, groups, rng.choice(["layer", "rms"]),
                       rng.choice(["none", "rms"]) if residual else "none", stream, block,
                       rng.choice(["f32", block]), rng.choice(["none", "f32", block]), residual,
                       rng.choice([1.0, 0.5, 1.4142135]) if residual else 1.0)
    else:
        head_dim = rng.choice([32, 64, 80, 96, 128, 256])
        heads = rng.randint(1, 5120 // head_dim)
        kv_heads = rng.choice([heads, heads, max(1, heads // 4), 1])
        batch = rng.choice([1, 1, 2, 3])
        T, H, W = rng.randint(1, 33), rng.randint(1, 64), rng.randint(1, 80)
        most = max(1, 75600 * 5120 // (batch * heads * head_dim) // 2)
        tokens = max(1, min(_log_int(rng, 1, T * H * W), most))
        positions = rng.choice(["grid", "listed"])
        x, out = rng.choice([("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("bf16", "f32"), ("f16", "f32")])
        c = _rope_case("", rng.choice(["fwd", "bwd"]), batch, T, H, W, tokens, rng.randint(0, T * H * W - tokens),
                       heads, kv_heads, head_dim, rng.choice(["none", "head", "token"]), x, out, rng.choice(["f32", x]),
                       positions, rng.choice(["interleaved", "halves"]), rng.choice(["axis", "shared"]),
                       rng.random() < 0.5, rng.choice([1e4, 1e6]))
    del c["name"]
    return c


# ------------------------------------------------------------------------------------------- inputs
def _randn(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _pair_table(c):
    """Per rotary pair: its axis and its angular frequency (double), for the default split of the pairs over
    the axes: c - 2 floor(c / 3), floor(c / 3), floor(c / 3) with c = head_dim / 2."""
    n = c["head_dim"] // 2
    third = n // 3
    counts = torch.tensor([n - 2 * third, third, third])
    axis = torch.repeat_interleave(torch.arange(3), counts)
    start = torch.repeat_interleave(torch.cumsum(counts, 0) - counts, counts)
    j = torch.arange(n)
    if c["schedule"] == "shared":
        power = j.double() / n
    else:
        power = (j - start).double() / counts[axis].double()
    return axis.cuda(), (float(c["theta"]) ** (-power)).cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "residual_norm":
        B, L, C, F = case["batch"], case["tokens"], case["channels"], case["groups"]
        stream, block, mod = _TYPES[case["stream"]], _TYPES[case["block"]], _TYPES[case["mod"]]
        # a residual stream: a mean off zero and a few channels an order of magnitude above the rest
        wide = 1.0 + 15.0 * (torch.rand(C, generator=g, device="cuda") < 0.01)
        s["x"] = _randn(g, (B, L, C), torch.float32).mul_(wide).add_(0.25).to(stream)
        s["y"] = _randn(g, (B, L, C), block) if case["residual"] else None
        s["gate"] = _randn(g, (B, F, C), mod, 0.5) if case["residual"] else None
        s["scale"] = _randn(g, (B, F, C), mod, 0.3)
        s["shift"] = _randn(g, (B, F, C), mod, 0.3)
        s["weight"] = s["bias"] = s["post_weight"] = None
        if case["weights"] != "none":
            wt = _TYPES[case["weights"]]
            s["weight"] = (1.0 + _randn(g, (C,), torch.float32, 0.1)).to(wt)
            if case["norm"] == "layer":
                s["bias"] = _randn(g, (C,), wt, 0.1)
            if case["post"] != "none":
                s["post_weight"] = (1.0 + _randn(g, (C,), torch.float32, 0.1)).to(wt)
        if case["direction"] == "bwd":
            s["dx_out"] = _randn(g, (B, L, C), stream, 0.1)
            s["dh"] = _randn(g, (B, L, C), block, 0.1)
    else:
        B, L, hq, hk, D = case["batch"], case["tokens"], case["heads"], case["kv_heads"], case["head_dim"]
        x, out, wt = _TYPES[case["x"]], _TYPES[case["out"]], _TYPES[case["weights"]]
        if case["fused"]:  # q and k as views of one projection's output [q | k | v]
            qkv = _randn(g, (B, L, hq + 2 * hk, D), x)
            s["q"], s["k"] = qkv[:, :, :hq], qkv[:, :, hq:hq + hk]
        else:
            s["q"], s["k"] = _randn(g, (B, L, hq, D), x), _randn(g, (B, L, hk, D), x)
        s["axis"], s["omega"] = _pair_table(case)
        s["wq"] = s["wk"] = s["positions"] = None
        if case["norm"] != "none":
            wide = 1 if case["norm"] == "head" else hq, 1 if case["norm"] == "head" else hk
            s["wq"] = (1.0 + _randn(g, (wide[0] * D,), torch.float32, 0.2)).to(wt)
            s["wk"] = (1.0 + _randn(g, (wide[1] * D,), torch.float32, 0.2)).to(wt)
        if case["positions"] == "listed":
            s["positions"] = torch.stack([torch.randint(0, n, (B, L), generator=g, device="cuda", dtype=torch.int32)
                                          for n in (case["T"], case["H"], case["W"])], dim=2).contiguous()
        if case["direction"] == "bwd":
            s["dq"], s["dk"] = _randn(g, (B, L, hq, D), out, 0.1), _randn(g, (B, L, hk, D), out, 0.1)
    return s


# ------------------------------------------------------------------------------- the framework's calls
def _own_residual_norm(s, c):
    from sparse_rank_hybrid_b200 import slra
    kinds = {"none": slra.NORM_NONE, "rms": slra.NORM_RMS, "layer": slra.NORM_LAYER}
    p = slra.ResidualNorm(c["batch"], c["tokens"], c["channels"], groups=c["groups"], norm=kinds[c["norm"]],
                          post_norm=kinds[c["post"]], residual_scale=c["residual_scale"])
    vectors = {n: s[n] for n in ("gate", "scale", "shift", "weight", "bias", "post_weight")}
    if c["direction"] == "fwd":
        # without a residual there is no y to give h its type
        x_out, h = slra.residual_norm_fwd(p, s["x"], s["y"], h_dtype=None if c["residual"] else _TYPES[c["block"]], **vectors)
        return [x_out, h] if c["residual"] else [h]
    g = slra.residual_norm_bwd(p, s["x"], s["y"], dh=s["dh"], dx_out=s["dx_out"], **vectors)
    return [t for t in (g.dx, g.dy, g.dgate, g.dscale, g.dshift, g.dweight, g.dbias, g.dpost_weight) if t is not None]


def _own_qk_rope(s, c):
    from sparse_rank_hybrid_b200 import slra
    p = slra.QkRope(c["batch"], c["tokens"], c["heads"], c["head_dim"], kv_heads=c["kv_heads"],
                    grid=(c["T"], c["H"], c["W"]), first_token=c["first"], theta=c["theta"],
                    norm={"none": slra.QK_NORM_NONE, "head": slra.QK_NORM_HEAD, "token": slra.QK_NORM_TOKEN}[c["norm"]],
                    pairing=slra.ROPE_HALVES if c["pairing"] == "halves" else slra.ROPE_INTERLEAVED,
                    schedule=slra.ROPE_SHARED if c["schedule"] == "shared" else slra.ROPE_PER_AXIS,
                    out_dtype={"bf16": slra.DTYPE_BF16, "f16": slra.DTYPE_F16, "f32": slra.DTYPE_F32}[c["out"]])
    if c["direction"] == "fwd":
        return list(slra.qk_rope_fwd(p, s["q"], s["k"], wq=s["wq"], wk=s["wk"], positions=s["positions"]))
    g = slra.qk_rope_bwd(p, s["q"], s["k"], s["dq"], s["dk"], wq=s["wq"], wk=s["wk"], positions=s["positions"])
    return [t for t in (g.dq, g.dk, g.dwq, g.dwk) if t is not None]


# -------------------------------------------------------------------------------------- plain forms
def _per_token(m, tokens):
    """A modulation [B, F, C] as [B, tokens, C] in fp32 (expanded, not copied, for one row per sample)."""
    m = m.float()
    return m if m.shape[1] in (1, tokens) else m.repeat_interleave(tokens // m.shape[1], dim=1)


def _per_group(g, groups):
    """A per-token gradient [B, L, C] summed over the tokens of each modulation row."""
    B, L, C = g.shape
    return g.view(B, groups, L // groups, C).sum(2)


def _plain_residual_norm(s, c):
    L, F, rs = c["tokens"], c["groups"], c["residual_scale"]
    stream, block = _TYPES[c["stream"]], _TYPES[c["block"]]
    x, eps = s["x"].float(), 1e-6
    if s["y"] is not None:
        gate = _per_token(s["gate"], L)
        y = s["y"].float()
        if c["post"] == "rms":
            ry = torch.rsqrt((y * y).mean(2, keepdim=True) + eps)
            y = y * ry
            if s["post_weight"] is not None:
                gate = gate * s["post_weight"].float()
        x = rs * x + gate * y
    mean = x.mean(2, keepdim=True) if c["norm"] == "layer" else 0.0
    n = x - mean
    rstd = torch.rsqrt((n * n).mean(2, keepdim=True) + eps)
    n = n * rstd
    w = s["weight"].float() if s["weight"] is not None else 1.0
    b = s["bias"].float() if s["bias"] is not None else 0.0
    up = 1.0 + _per_token(s["scale"], L)
    if c["direction"] == "fwd":
        h = ((n * w + b) * up + _per_token(s["shift"], L)).to(block)
        return [x.to(stream), h] if s["y"] is not None else [h]
    dh = s["dh"].float()
    out_scale, out_shift = _per_group(dh * (n * w + b), F), _per_group(dh, F)
    dn = dh * up
    dweight = (dn * n).sum((0, 1)) if s["weight"] is not None else None
    dbias = dn.sum((0, 1)) if s["bias"] is not None else None
    dn = dn * w
    dx = dn - n * (dn * n).mean(2, keepdim=True)
    if c["norm"] == "layer":
        dx = dx - dn.mean(2, keepdim=True)
    dx = s["dx_out"].float() + dx * rstd
    if s["y"] is None:
        return [t for t in (dx.to(stream), out_scale, out_shift, dweight, dbias) if t is not None]
    through = dx * y
    dpost = None
    if s["post_weight"] is not None:
        dgate = _per_group(through * s["post_weight"].float(), F)
        dpost = (through * _per_token(s["gate"], L)).sum((0, 1))
    else:
        dgate = _per_group(through, F)
    dy = dx * gate
    if c["post"] == "rms":
        dy = ry * (dy - y * (dy * y).mean(2, keepdim=True))
    grads = ((rs * dx).to(stream), dy.to(block), dgate, out_scale, out_shift, dweight, dbias, dpost)
    return [t for t in grads if t is not None]


def _token_positions(s, c):
    """int64 [B or 1, L, 3] positions along (t, h, w)."""
    if s["positions"] is not None:
        return s["positions"].long()
    n = torch.arange(c["first"], c["first"] + c["tokens"], device="cuda")
    return torch.stack([n // (c["H"] * c["W"]), (n // c["W"]) % c["H"], n % c["W"]], dim=1)[None]


def _turn(x, cos, sin, halves):
    """x [B, L, heads, D] rotated pair by pair; cos, sin [B or 1, L, 1, D / 2]."""
    half = x.shape[3] // 2
    if halves:
        a, b = x[..., :half], x[..., half:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos], dim=3)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cos - b * sin, a * sin + b * cos], dim=4).flatten(3)


def _plain_one(x, w, c, cos, sin, d):
    """One of q, k: its rotated norm, or the gradients of x and of the weight from d."""
    halves, eps = c["pairing"] == "halves", 1e-6
    dims = {"none": None, "head": (3,), "token": (2, 3)}[c["norm"]]
    out_type = _TYPES[c["out"]]
    xf = x.float()
    n, wf = xf, None
    if dims:
        r = torch.rsqrt((xf * xf).mean(dims, keepdim=True) + eps)
        n = xf * r
        wf = w.float().view(-1, x.shape[3])
    if d is None:
        return _turn(n if wf is None else n * wf, cos, sin, halves).to(out_type), None
    dn = _turn(d.float(), cos, -sin, halves)
    if wf is None:
        return dn.to(x.dtype), None
    dw = (dn * n).sum((0, 1, 2) if c["norm"] == "head" else (0, 1)).flatten()
    dn = dn * wf
    return (r * (dn - n * (dn * n).mean(dims, keepdim=True))).to(x.dtype), dw


def _plain_qk_rope(s, c):
    angle = _token_positions(s, c)[..., s["axis"]].double() * s["omega"]
    cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]
    q, dwq = _plain_one(s["q"], s["wq"], c, cos, sin, s.get("dq"))
    k, dwk = _plain_one(s["k"], s["wk"], c, cos, sin, s.get("dk"))
    return [t for t in (q, k, dwq, dwk) if t is not None]


def run(state):
    c = state["case"]
    if own:
        return _own_residual_norm(state, c) if c["op"] == "residual_norm" else _own_qk_rope(state, c)
    return _plain_residual_norm(state, c) if c["op"] == "residual_norm" else _plain_qk_rope(state, c)


# --------------------------------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "residual_norm":
        rows, C = c["batch"] * c["tokens"], c["channels"]
        S, K, M = _BYTES[c["stream"]], _BYTES[c["block"]], _BYTES[c["mod"]]
        mods = c["batch"] * c["groups"] * C
        weights = 0 if c["weights"] == "none" else (1 + (c["norm"] == "layer") + (c["post"] != "none")) * C
        wb = _BYTES.get(c["weights"], 0)
        vectors = mods * M * (3 if c["residual"] else 2) + weights * wb
        if c["direction"] == "fwd":
            # x, y in; x_out, h out
            per = 2 * S + 2 * K if c["residual"] else S + K
            return {"bytes": rows * C * per + vectors, "flops": rows * C * (12 if c["residual"] else 8)}
        # x, y, dx_out, dh in; dx, dy out; the vectors' gradients in fp32
        per = 3 * S + 3 * K if c["residual"] else 3 * S + K
        vectors += 4 * (mods * (3 if c["residual"] else 2) + weights)
        return {"bytes": rows * C * per + vectors, "flops": rows * C * (30 if c["residual"] else 20)}
    rows, D = c["batch"] * c["tokens"], c["head_dim"]
    heads = c["heads"] + c["kv_heads"]
    X, O = _BYTES[c["x"]], _BYTES[c["out"]]
    weights = {"none": 0, "head": 2 * D, "token": heads * D}[c["norm"]]
    listed_positions = rows * 12 if c["positions"] == "listed" else 0
    if c["direction"] == "fwd":
        return {"bytes": rows * heads * D * (X + O) + weights * _BYTES[c["weights"]] + listed_positions,
                "flops": rows * heads * D * (3 if c["norm"] == "none" else 7)}
    # x and the gradient in, dx out (without a norm x itself is not needed); the weights' gradients in fp32
    per = X + O if c["norm"] == "none" else 2 * X + O
    return {"bytes": rows * heads * D * per + weights * (_BYTES[c["weights"]] + 4) + listed_positions,
            "flops": rows * heads * D * (3 if c["norm"] == "none" else 14)}


# ------------------------------------------------------------------------------------ the definition
def _exact_residual_norm(s, c):
    """Token ranges through the definition in double, the gradients by autograd."""
    B, L, C, F, rs = c["batch"], c["tokens"], c["channels"], c["groups"], c["residual_scale"]
    backward = c["direction"] == "bwd"
    leaf = {n: None if s[n] is None else s[n].double().requires_grad_(backward)
            for n in ("gate", "scale", "shift", "weight", "bias", "post_weight")}

    def norm(v, kind, weight, bias):
        if kind == "none":
            return v
        if kind == "layer":
            v = v - v.sum(1, keepdim=True) / C
        v = v / torch.sqrt((v ** 2).sum(1, keepdim=True) / C + 1e-6)
        v = v if weight is None else v * weight
        return v if bias is None else v + bias

    x_out, h, dx, dy = [], [], [], []
    step = max(1, (1 << 24) // C)
    for b in range(B):
        for lo in range(0, L, step):
            hi = min(L, lo + step)
            row = torch.arange(lo, hi, device="cuda") // (L // F)
            x = s["x"][b, lo:hi].double().requires_grad_(backward)
            y = None if s["y"] is None else s["y"][b, lo:hi].double().requires_grad_(backward)
            o = x
            if y is not None:
                o = rs * x + leaf["gate"][b, row] * norm(y, c["post"], leaf["post_weight"], None)
            r = norm(o, c["norm"], leaf["weight"], leaf["bias"]) * (1 + leaf["scale"][b, row]) + leaf["shift"][b, row]
            if backward:
                ((r * s["dh"][b, lo:hi].double()).sum() + (o * s["dx_out"][b, lo:hi].double()).sum()).backward()
                dx.append(x.grad)
                dy.append(None if y is None else y.grad)
            else:
                x_out.append(o)
                h.append(r)

    def whole(parts):
        return torch.cat(parts).view(B, L, C)

    if not backward:
        return [whole(x_out), whole(h)] if c["residual"] else [whole(h)]
    first = [whole(dx)] + ([whole(dy)] if c["residual"] else [])
    names = (["gate"] if c["residual"] else []) + ["scale", "shift", "weight", "bias", "post_weight"]
    return first + [leaf[n].grad for n in names if leaf[n] is not None]


def _exact_qk_rope(s, c):
    """Pairs as complex numbers times exp(i angle) in double, token ranges, the gradients by autograd."""
    B, L, D = c["batch"], c["tokens"], c["head_dim"]
    n, backward = D // 2, c["direction"] == "bwd"
    counts = [n - 2 * (n // 3), n // 3, n // 3]
    schedule = [(a, float(c["theta"]) ** (-((m if c["schedule"] == "axis" else sum(counts[:a]) + m)
                                           / (counts[a] if c["schedule"] == "axis" else n))))
                for a in range(3) for m in range(counts[a])]
    axes = torch.tensor([a for a, _ in schedule], device="cuda")
    omega = torch.tensor([f for _, f in schedule], device="cuda", dtype=torch.float64)
    outs, weight_grads = [], []
    for x_all, w, d_all in ((s["q"], s["wq"], s.get("dq")), (s["k"], s["wk"], s.get("dk"))):
        heads = x_all.shape[2]
        weight = None if w is None else w.double().requires_grad_(backward)
        parts = []
        step = max(1, (1 << 23) // (heads * D))
        for b in range(B):
            for lo in range(0, L, step):
                hi = min(L, lo + step)
                if s["positions"] is not None:
                    at = s["positions"][b, lo:hi].double()
                else:
                    token = torch.arange(c["first"] + lo, c["first"] + hi, device="cuda")
                    rest = token % (c["H"] * c["W"])
                    at = torch.stack([(token - rest) // (c["H"] * c["W"]), rest // c["W"], rest % c["W"]], 1).double()
                turn = torch.polar(torch.ones((), device="cuda", dtype=torch.float64), at[:, axes] * omega)[:, None]
                x = x_all[b, lo:hi].double().requires_grad_(backward)
                v = x
                if c["norm"] == "head":
                    v = v / torch.sqrt((v ** 2).sum(2, keepdim=True) / D + 1e-6) * weight
                elif c["norm"] == "token":
                    v = v / torch.sqrt((v ** 2).sum((1, 2), keepdim=True) / (heads * D) + 1e-6) * weight.view(heads, D)
                if c["pairing"] == "halves":
                    z = torch.complex(v[..., :n].contiguous(), v[..., n:].contiguous()) * turn
                    v = torch.cat([z.real, z.imag], 2)
                else:
                    v = torch.view_as_real(torch.view_as_complex(v.reshape(hi - lo, heads, n, 2)) * turn).flatten(2)
                if backward:
                    (v * d_all[b, lo:hi].double()).sum().backward()
                    parts.append(x.grad)
                else:
                    parts.append(v)
        outs.append(torch.cat(parts).view(B, L, heads, D))
        if backward and weight is not None:
            weight_grads.append(weight.grad)
    return outs + weight_grads


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_residual_norm(s, case) if case["op"] == "residual_norm" else _exact_qk_rope(s, case)
