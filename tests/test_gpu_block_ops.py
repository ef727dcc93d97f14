"""The operators around the attention on the GPU: residual_norm and qk_rope, forward and backward.

Each output is compared element by element with the definition in double.  The tolerance is derived from
the arithmetic: half a step of the output's type relative to the value, plus K roundings of fp32 (2^-24
each) of an elementwise bound M on the terms that meet in the value.  K = 64 covers a row: about twenty
additions of a sum over the row (eight in a thread, five shuffles each within and across warps), the
products before and after it, rsqrt and sincospi.  M carries the one amplification there is: a centred
value o - m inherits the error of o and m, of relative size rho = rms(|o| + |m|) / std.  Sums over tokens
add one rounding per row of a worker (at most ceil(rows / 148) rows) to that.
"""
import math

import pytest
import torch

from sparse_rank_hybrid_b200 import slra

pytestmark = pytest.mark.gpu

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
U32 = 2.0 ** -24
K_ROW = 64


@pytest.fixture(scope="module", autouse=True)
def _build():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from sparse_rank_hybrid_b200 import build
    build.build()


def close(got, ref, M, label, k=K_ROW):
    """|got - ref| <= half a step of got's type at ref + k fp32 roundings of M (+ the type's subnormal step)."""
    fi = torch.finfo(got.dtype)
    tol = fi.eps / 2 * ref.abs() + k * U32 * M * (1 + fi.eps) + fi.tiny * fi.eps
    err = (got.double() - ref).abs()
    worst = float((err / tol).max())
    assert bool((err <= tol).all()), f"{label}: {worst:.3g} times the tolerance"
    return worst


def rnd(g, shape, dtype, std=1.0, mean=0.0):
    return (torch.randn(shape, generator=g, device="cuda") * std + mean).to(dtype)


# ------------------------------------------------------------------------------------ residual norm
def norm_inputs(B, L, C, F=1, stream=BF, block=BF, mod=FP, weights=None, norm=slra.NORM_LAYER, post=slra.NORM_NONE,
                residual=True, rs=1.0, seed=0, mean=0.25):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = {"x": rnd(g, (B, L, C), stream, 1.0, mean), "y": rnd(g, (B, L, C), block) if residual else None,
         "gate": rnd(g, (B, F, C), mod, 0.5) if residual else None,
         "scale": rnd(g, (B, F, C), mod, 0.3), "shift": rnd(g, (B, F, C), mod, 0.3),
         "weight": None, "bias": None, "post_weight": None}
    if norm == slra.NORM_NONE:
        t["scale"] = t["shift"] = None
    elif weights is not None:
        t["weight"] = rnd(g, (C,), weights, 0.2, 1.0)
        if norm == slra.NORM_LAYER:
            t["bias"] = rnd(g, (C,), weights, 0.2)
    if weights is not None and post != slra.NORM_NONE:
        t["post_weight"] = rnd(g, (C,), weights, 0.2, 1.0)
    p = slra.ResidualNorm(B, L, C, groups=F, norm=norm, post_norm=post, residual_scale=rs)
    d = {"dh": rnd(g, (B, L, C), block, 0.1) if norm != slra.NORM_NONE else None, "dx_out": rnd(g, (B, L, C), stream, 0.1)}
    return p, t, d


def norm_reference(p, t, d=None):
    """Every output of the definition in double, with its bound M: {name: (value, M)}."""
    B, L, C, F = p.batch, p.tokens, p.channels, p.groups
    dbl = {n: None if v is None else v.double() for n, v in t.items()}

    def per_token(m, fill):
        return torch.full((1, 1, 1), fill, device="cuda", dtype=torch.float64) if m is None else \
            m.repeat_interleave(L // F, dim=1)

    def vec(v, fill):
        return torch.full((1,), fill, device="cuda", dtype=torch.float64) if v is None else v

    x, y = dbl["x"], dbl["y"]
    scale, shift, gate = (per_token(dbl[n], f) for n, f in (("scale", 0.0), ("shift", 0.0), ("gate", 1.0)))
    w, b, wp = vec(dbl["weight"], 1.0), vec(dbl["bias"], 0.0), vec(dbl["post_weight"], 1.0)
    o, Mo, ry, yh = x, x.abs(), 1.0, None
    if y is not None:
        ry = torch.rsqrt((y * y).mean(2, keepdim=True) + p.post_eps) if p.post_norm else torch.ones_like(x[..., :1])
        yh = y * ry
        G = gate * wp
        o = p.residual_scale * x + G * yh
        Mo = (p.residual_scale * x).abs() + (G * yh).abs()
    out = {"x_out": (o, Mo)}
    if p.norm:
        m = o.mean(2, keepdim=True) if p.norm == slra.NORM_LAYER else torch.zeros_like(o[..., :1])
        Mm = Mo.mean(2, keepdim=True) if p.norm == slra.NORM_LAYER else torch.zeros_like(o[..., :1])
        r = torch.rsqrt(((o - m) ** 2).mean(2, keepdim=True) + p.eps)
        n = (o - m) * r
        rho = ((Mo + Mm) ** 2).mean(2, keepdim=True).sqrt() * r
        Nm = r * (Mo + Mm) + n.abs() * rho
        A = w * (1 + scale)
        out["h"] = (n * A + b * (1 + scale) + shift, Nm * A.abs() + (b * (1 + scale)).abs() + shift.abs())
    if d is None:
        return out
    dxo = torch.zeros_like(x) if d["dx_out"] is None else d["dx_out"].double()
    tt, Mt = dxo, dxo.abs()
    if p.norm:
        dh = d["dh"].double()
        a = dh * A
        am = a.mean(2, keepdim=True) if p.norm == slra.NORM_LAYER else 0.0
        tt = dxo + r * (a - am - n * (a * n).mean(2, keepdim=True))
        Mt = dxo.abs() + r * (1 + rho) * (a.abs() + a.abs().mean(2, keepdim=True) + Nm * (a.abs() * Nm).mean(2, keepdim=True))
    out["dx"] = (p.residual_scale * tt, abs(p.residual_scale) * Mt)

    def grouped(v):
        return v.expand(B, L, C).reshape(B, F, L // F, C).sum(2)

    def total(v):
        return v.expand(B, L, C).sum((0, 1))

    if p.norm:
        if t["scale"] is not None:
            out["dscale"] = (grouped(dh * (n * w + b)), grouped(dh.abs() * (Nm * w.abs() + b.abs())))
        if t["shift"] is not None:
            out["dshift"] = (grouped(dh), grouped(dh.abs()))
        if t["weight"] is not None:
            out["dweight"] = (total(dh * (1 + scale) * n), total(dh.abs() * (1 + scale).abs() * Nm))
        if t["bias"] is not None:
            out["dbias"] = (total(dh * (1 + scale)), total(dh.abs() * (1 + scale).abs()))
    if y is not None:
        u, Mu = tt * G, Mt * G.abs()
        if p.post_norm:
            out["dy"] = (ry * (u - yh * (u * yh).mean(2, keepdim=True)),
                         ry * (Mu + yh.abs() * (Mu * yh.abs()).mean(2, keepdim=True)))
        else:
            out["dy"] = (u, Mu)
        if t["gate"] is not None:
            out["dgate"] = (grouped(tt * yh * wp), grouped(Mt * (yh * wp).abs()))
        if t["post_weight"] is not None:
            out["dpost_weight"] = (total(tt * gate * yh), total(Mt * (gate * yh).abs()))
    return out


def check_norm_forward(p, t):
    x_out, h = slra.residual_norm_fwd(p, **t)
    ref = norm_reference(p, t)
    if t["y"] is not None:
        close(x_out, *ref["x_out"], "x_out")
    if p.norm:
        close(h, *ref["h"], "h")


def check_norm_backward(p, t, d, **kw):
    got = slra.residual_norm_bwd(p, **t, **d, **kw)
    ref = norm_reference(p, t, d)
    rows = K_ROW + -(-p.batch * p.tokens // 148)
    for name in ("dx", "dy", "dgate", "dscale", "dshift", "dweight", "dbias", "dpost_weight"):
        g = getattr(got, name)
        assert (g is not None) == (name in ref), name
        if g is not None:
            close(g, *ref[name], name, K_ROW if name in ("dx", "dy") else rows)
    return got


# rows from one to several a worker, channels within a warp, over several warps, two vectors a thread
SIZES = [(1, 1, 8), (1, 1, 1536), (700, 1, 48), (500, 2, 1536), (2, 3, 24), (1, 37, 256), (3, 41, 264), (2, 150, 1032), (1, 700, 1536), (1, 5, 5120),
         (1, 301, 5128), (1, 9, 8192), (5, 401, 64)]
TYPES = [(BF, BF), (FP, BF), (HF, HF), (FP, HF), (FP, FP)]


@pytest.mark.parametrize("B,L,C", SIZES)
def test_norm_sizes(B, L, C):
    p, t, d = norm_inputs(B, L, C, seed=C + L)
    check_norm_forward(p, t)
    check_norm_backward(p, t, d)


@pytest.mark.parametrize("stream,block", TYPES)
@pytest.mark.parametrize("C", [72, 640, 6000])
def test_norm_types(stream, block, C):
    for mod in {FP, block}:
        p, t, d = norm_inputs(2, 33, C, 3, stream, block, mod, weights=block, post=slra.NORM_RMS, rs=0.5, seed=C)
        check_norm_forward(p, t)
        check_norm_backward(p, t, d)


@pytest.mark.parametrize("stream,block", TYPES)
def test_norm_widest_rows(stream, block):
    """8192 channels: one step of the ring for fp32, the weights' sums outside shared memory."""
    p, t, d = norm_inputs(1, 300, 8192, 2, stream, block, weights=FP, post=slra.NORM_RMS, seed=40)
    check_norm_forward(p, t)
    check_norm_backward(p, t, d)


@pytest.mark.parametrize("mod", [BF, HF, FP])
@pytest.mark.parametrize("weights", [BF, HF, FP])
@pytest.mark.parametrize("stream", [FP, BF])
def test_norm_vector_types(mod, weights, stream):
    """Modulation and weights of any type, whatever the rows'."""
    p, t, d = norm_inputs(2, 14, 152, 2, stream, BF, mod, weights=weights, post=slra.NORM_RMS, seed=41)
    check_norm_forward(p, t)
    check_norm_backward(p, t, d)


@pytest.mark.parametrize("rs", [0.0, -2.0, 1e-3])
def test_norm_residual_scale(rs):
    p, t, d = norm_inputs(1, 40, 512, rs=rs, seed=42)
    check_norm_forward(p, t)
    check_norm_backward(p, t, d)


@pytest.mark.parametrize("norm", [slra.NORM_NONE, slra.NORM_RMS, slra.NORM_LAYER])
@pytest.mark.parametrize("post", [slra.NORM_NONE, slra.NORM_RMS])
@pytest.mark.parametrize("weights", [None, FP])
@pytest.mark.parametrize("residual", [True, False])
def test_norm_options(norm, post, weights, residual):
    if not residual and (norm == slra.NORM_NONE or post != slra.NORM_NONE):
        pytest.skip("nothing to compute")
    p, t, d = norm_inputs(2, 21, 400, 1, weights=weights, norm=norm, post=post, residual=residual, seed=3,
                          rs=1.25 if residual else 1.0)
    check_norm_forward(p, t)
    check_norm_backward(p, t, d)
    check_norm_backward(p, t, dict(d, dx_out=None))


@pytest.mark.parametrize("B,L,F,C", [(1, 21 * 13, 21, 1536), (3, 28, 7, 200), (2, 50, 50, 64), (1, 400, 400, 1536),
                                     (2, 900, 450, 320), (1, 2000, 2, 72), (4, 1, 1, 640), (1, 1000, 1000, 5128)])
@pytest.mark.parametrize("weights", [None, BF])
def test_norm_modulation_rows(B, L, F, C, weights):
    """One modulation row per sample, frame or token; workers that share a row, and rows inside a worker."""
    p, t, d = norm_inputs(B, L, C, F, weights=weights, post=slra.NORM_RMS if weights else slra.NORM_NONE, seed=F)
    check_norm_forward(p, t)
    check_norm_backward(p, t, d)


@pytest.mark.parametrize("stream,block", TYPES)
@pytest.mark.parametrize("B,L,C", [(3, 4001, 72), (5, 1300, 240), (3, 1333, 392), (2, 700, 1536), (2, 307, 5120), (1, 450, 5136),
                                   (1, 300, 8192)])
def test_norm_modulation_for_each_token(stream, block, B, L, C):
    """Several rows a worker with vectors of their own: rings of several stages, and rows too wide for two."""
    for mod, weights, norm, post in ((FP, FP, slra.NORM_LAYER, slra.NORM_RMS), (block, block, slra.NORM_RMS, slra.NORM_NONE),
                                     (block, None, slra.NORM_LAYER, slra.NORM_NONE)):
        p, t, d = norm_inputs(B, L, C, L, stream, block, mod, weights=weights, norm=norm, post=post, rs=0.5, seed=C)
        check_norm_forward(p, t)
        check_norm_backward(p, t, d)


@pytest.mark.parametrize("F", [1, 5930])
@pytest.mark.parametrize("C", [2568, 3336, 4096])
def test_norm_two_vectors_a_thread(C, F):
    """Many 16-bit rows of about half a block's channels."""
    for post in (slra.NORM_NONE, slra.NORM_RMS):
        p, t, d = norm_inputs(1, 5930, C, F, HF, HF, HF, weights=FP, post=post, seed=47)
        check_norm_backward(p, t, d)


@pytest.mark.parametrize("C", [88, 1040])
@pytest.mark.parametrize("given", [("gate",), ("scale",), ("shift",), ("gate", "shift", "weight"), ("scale", "bias"), ("post_weight",)])
def test_norm_some_vectors_for_each_token(C, given):
    p, t, d = norm_inputs(2, 800, C, 800, stream=FP, weights=BF, post=slra.NORM_RMS, seed=43)
    for n in ("gate", "scale", "shift", "weight", "bias", "post_weight"):
        if n not in given:
            t[n] = None
    check_norm_forward(p, t)
    check_norm_backward(p, t, d)


def test_norm_vectors_for_each_token_broadcast_and_strided():
    """Rows of a wider tensor, and one row behind every token and sample."""
    for C in (88, 1040):
        p, t, d = norm_inputs(3, 500, C, 500, stream=FP, weights=BF, seed=44)
        wide = torch.randn(3, 500, 3 * C, device="cuda")
        t["gate"], t["scale"] = wide[:, :, :C], wide[:, :, 2 * C:]
        t["shift"] = wide[:1, :1, C:2 * C].expand(3, 500, C)
        check_norm_forward(p, t)
        check_norm_backward(p, t, d)


def test_norm_without_residual_for_each_token():
    for C in (88, 1040):
        p, t, d = norm_inputs(2, 600, C, 600, stream=HF, block=HF, mod=HF, weights=HF, residual=False, seed=45)
        check_norm_forward(p, t)
        check_norm_backward(p, t, d)


@pytest.mark.parametrize("B,L,F,C", [(1, 20000, 1, 64), (2, 9000, 3, 392), (1, 3000, 1, 1536), (1, 3000, 30, 1536), (40, 50, 1, 136),
                                     (1, 600, 1, 5128)])
def test_norm_many_partial_sums(B, L, F, C):
    """Joins over one warp, a block and a cluster, of few columns and of many; twice with the same bits."""
    p, t, d = norm_inputs(B, L, C, F, weights=FP, post=slra.NORM_RMS, seed=46)
    one = check_norm_backward(p, t, d)
    two = slra.residual_norm_bwd(p, **t, **d)
    for a, b in zip(one[:8], two[:8]):
        assert a is None or torch.equal(a, b)


def test_norm_without_vectors():
    for given in ((), ("gate",), ("scale",), ("shift",), ("weight",), ("bias",), ("post_weight",)):
        p, t, d = norm_inputs(2, 19, 136, weights=FP, post=slra.NORM_RMS, seed=5)
        for n in ("gate", "scale", "shift", "weight", "bias", "post_weight"):
            if n not in given:
                t[n] = None
        check_norm_forward(p, t)
        check_norm_backward(p, t, d)


@pytest.mark.parametrize("mean", [0.0, 100.0, 1000.0])
def test_norm_mean_far_from_zero(mean):
    """The variance of rows whose mean is far above their spread."""
    p, t, d = norm_inputs(1, 64, 1536, stream=FP, seed=8, mean=mean)
    check_norm_forward(p, t)
    check_norm_backward(p, t, d)


@pytest.mark.parametrize("C", [64, 1536])
def test_norm_rows_of_zeros_infinities_and_nan(C):
    """A row of zeros gives the shift; a row with an infinity or NaN gives NaN in h and leaves its neighbours."""
    p, t, _ = norm_inputs(1, 9, C, seed=9)
    t["x"][0, 2] = 0
    t["y"][0, 2] = 0
    t["x"][0, 4, 3] = float("inf")
    t["y"][0, 6, 5] = float("nan")
    x_out, h = slra.residual_norm_fwd(p, **t)
    assert torch.equal(h[0, 2], t["shift"][0, 0].to(BF)) and not x_out[0, 2].any()
    assert h[0, 4].isnan().all() and h[0, 6].isnan().all()
    assert x_out[0, 4, 3] == float("inf") and x_out[0, 6, 5].isnan() and x_out[0, 6].isnan().sum() == 1
    keep = [0, 1, 2, 3, 5, 7, 8]
    clean = dict(t, x=t["x"].clone(), y=t["y"].clone())
    clean["x"][0, 4, 3] = clean["y"][0, 6, 5] = 0
    ref = slra.residual_norm_fwd(p, **clean)
    assert torch.equal(x_out[0, keep], ref[0][0, keep]) and torch.equal(h[0, keep], ref[1][0, keep])


def test_norm_strides_broadcasts_and_in_place():
    p, t, d = norm_inputs(2, 30, 320, 3, stream=FP, seed=10)
    x_out, h = slra.residual_norm_fwd(p, **t)
    ref = slra.residual_norm_bwd(p, **t, **d)

    def wide(v, fill=7.0):  # rows of a wider buffer, batch and token order swapped
        buf = torch.full((v.shape[1], v.shape[0], v.shape[2] + 16), fill, dtype=v.dtype, device="cuda")
        view = buf[:, :, 8:8 + v.shape[2]].transpose(0, 1)
        view.copy_(v)
        return buf, view

    s = {n: wide(t[n])[1] for n in ("x", "y")}
    mods = torch.stack([t["gate"], t["scale"], t["shift"]], dim=1).contiguous()  # [B, 3, F, C] as one projection
    m = {n: mods[:, i] for i, n in enumerate(("gate", "scale", "shift"))}
    (bo, vo), (bh, vh) = wide(torch.zeros_like(x_out)), wide(torch.zeros_like(h))
    got = slra.residual_norm_fwd(p, s["x"], s["y"], **m, x_out=vo, h=vh)
    assert got[0] is vo and torch.equal(vo, x_out) and torch.equal(vh, h)
    for buf in (bo, bh):  # nothing outside the rows was touched
        assert (buf[:, :, :8] == 7).all() and (buf[:, :, -8:] == 7).all()
    (bx, vx), (by, vy) = wide(torch.zeros_like(ref.dx)), wide(torch.zeros_like(ref.dy))
    g = slra.residual_norm_bwd(p, s["x"], s["y"], dh=wide(d["dh"])[1], dx_out=wide(d["dx_out"])[1], **m, dx=vx, dy=vy)
    assert torch.equal(vx, ref.dx) and torch.equal(vy, ref.dy)
    assert (bx[:, :, :8] == 7).all() and (by[:, :, -8:] == 7).all()
    for n in ("dgate", "dscale", "dshift"):
        assert torch.equal(getattr(g, n), getattr(ref, n))
    # in place: x_out over x, h over y, dx over dx_out, dy over dh
    x, y = t["x"].clone(), t["y"].clone()
    got = slra.residual_norm_fwd(p, x, y, t["gate"], t["scale"], t["shift"], x_out=x, h=y)
    assert torch.equal(x, x_out) and torch.equal(y, h)
    dx, dy = d["dx_out"].clone(), d["dh"].clone()
    slra.residual_norm_bwd(p, **t, dh=dy, dx_out=dx, dx=dx, dy=dy)
    assert torch.equal(dx, ref.dx) and torch.equal(dy, ref.dy)
    # one modulation row for everything, as an expanded view: gradients still per sample and row
    one = {n: t[n][:1, :1].expand(2, 3, 320) for n in ("gate", "scale", "shift")}
    full = {n: v.contiguous() for n, v in one.items()}
    a, b = slra.residual_norm_fwd(p, t["x"], t["y"], **one), slra.residual_norm_fwd(p, t["x"], t["y"], **full)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga, gb = (slra.residual_norm_bwd(p, t["x"], t["y"], **d, **m_) for m_ in (one, full))
    assert all(torch.equal(getattr(ga, n), getattr(gb, n)) for n in ("dx", "dy", "dgate", "dscale", "dshift"))


def test_offsets_past_32_bits():
    """Rows and heads more than 2^31 elements apart: the same bits as packed ones."""
    far = 2 ** 30 + 8
    buf = torch.zeros(2 * far + 4096, dtype=BF, device="cuda")
    p, t, _ = norm_inputs(1, 3, 1024, seed=30)
    x = buf.as_strided((1, 3, 1024), (3 * far, far, 1))
    x.copy_(t["x"])
    ref = slra.residual_norm_fwd(p, **t)
    got = slra.residual_norm_fwd(p, **dict(t, x=x), x_out=x)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    rp, rt, _ = rope_inputs(3, 1, 8, 0, 128, seed=31)
    q = buf.as_strided((3, 1, 8, 128), (far, 1024, 128, 1))
    q.copy_(rt["q"])
    out = slra.qk_rope_fwd(rp, q, wq=rt["wq"], out_q=q)[0]
    assert out is q and torch.equal(q, slra.qk_rope_fwd(rp, **rt)[0])


def test_calls_on_two_streams_at_once():
    """Calls that overlap on the GPU share nothing: each gives its own bits."""
    cases = []
    for seed in (0, 1):
        p, t, d = norm_inputs(1, 3000, 640, 3, weights=FP, seed=seed)
        rp, rt, rd = rope_inputs(1, 3000, 5, 5, 128, norm=slra.QK_NORM_TOKEN, seed=seed)
        ref = (*slra.residual_norm_bwd(p, **t, **d)[:7], *slra.qk_rope_bwd(rp, rt["q"], rt["k"], **rd, wq=rt["wq"], wk=rt["wk"])[:4])
        cases.append((p, t, d, rp, rt, rd, ref, torch.cuda.Stream()))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, (p, t, d, rp, rt, rd, _, s) in enumerate(cases):
            a = slra.residual_norm_bwd(p, **t, **d, stream=s)
            b = slra.qk_rope_bwd(rp, rt["q"], rt["k"], **rd, wq=rt["wq"], wk=rt["wk"], stream=s)
            got[i].append((*a[:7], *b[:4]))
    torch.cuda.synchronize()
    for i in (0, 1):
        for run in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(run, cases[i][6]))


def test_norm_first_block_types():
    """Without y the norm's output type is free beside an fp32 stream."""
    p, t, _ = norm_inputs(1, 13, 128, stream=FP, residual=False, seed=11)
    x, h = slra.residual_norm_fwd(p, t["x"], scale=t["scale"], shift=t["shift"], h_dtype=BF)
    assert x is t["x"] and h.dtype is BF
    close(h, *norm_reference(p, t)["h"], "h")


def test_norm_gradients_against_differences():
    """The gradients against central differences of the definition, each input along a random direction.
    Step e = 1e-4 of the double definition: truncation ~ e^2 of the third derivative, ~1e-7 of the slope for
    unit-scale rows; the kernel's fp32 gradients add 64 roundings of the slope's terms."""
    p, t, d = norm_inputs(2, 12, 64, 2, FP, FP, FP, weights=FP, post=slra.NORM_RMS, rs=0.75, seed=12)
    g = slra.residual_norm_bwd(p, **t, **d)

    def loss(tt):
        r = norm_reference(p, tt)
        return float((r["x_out"][0] * d["dx_out"].double()).sum() + (r["h"][0] * d["dh"].double()).sum())

    gen = torch.Generator(device="cuda").manual_seed(1)
    for name in ("x", "y", "gate", "scale", "shift", "weight", "bias", "post_weight"):
        v = torch.randn(t[name].shape, generator=gen, device="cuda", dtype=torch.float64)
        e = 1e-4
        slope = (loss(dict(t, **{name: t[name].double() + e * v})) - loss(dict(t, **{name: t[name].double() - e * v}))) / (2 * e)
        terms = getattr(g, "d" + name).double() * v
        assert abs(float(terms.sum()) - slope) <= 1e-5 * float(terms.abs().sum()), name


def test_norm_deterministic_streams_and_graphs():
    """Same bits run after run; on another stream; from a captured graph replayed on new inputs, two graphs
    sharing one workspace; with the library's own workspace."""
    import ctypes
    p, t, d = norm_inputs(1, 2000, 640, 5, weights=FP, post=slra.NORM_RMS, seed=13)
    ref = slra.residual_norm_bwd(p, **t, **d)
    names = [n for n in ref._fields if n != "workspace"]
    ws = ref.workspace
    again = slra.residual_norm_bwd(p, **t, **d, workspace=ws)
    assert again.workspace is ws and all(torch.equal(getattr(again, n), getattr(ref, n)) for n in names)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = slra.residual_norm_bwd(p, **t, **d, stream=s)
    f_other = slra.residual_norm_fwd(p, **t, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    f = slra.residual_norm_fwd(p, **t)
    assert all(torch.equal(getattr(other, n), getattr(ref, n)) for n in names)
    assert torch.equal(f[0], f_other[0]) and torch.equal(f[1], f_other[1])
    # the library's own workspace: NULL
    c = slra._residual_norm_problem(p, t["x"], t["y"], d["dh"], *(t[n] for n in ("gate", "scale", "shift", "weight",
                                                                                  "bias", "post_weight")))[0]
    own = {n: torch.empty_like(getattr(ref, n)) for n in names}
    for n in names[2:]:
        setattr(c, n, own[n].data_ptr())
    assert slra.lib().slra_residual_norm_bwd(ctypes.byref(c), t["x"].data_ptr(), t["y"].data_ptr(), d["dx_out"].data_ptr(),
                                             d["dh"].data_ptr(), own["dx"].data_ptr(), own["dy"].data_ptr(), None, 0,
                                             torch.cuda.current_stream().cuda_stream) == slra.OK
    assert all(torch.equal(own[n], getattr(ref, n)) for n in names)
    # graphs: with the workspace given, with one of the binding's, with one of the library's
    torch.cuda.synchronize()
    graphs = []
    for w in (ws, ws, None):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = (slra.residual_norm_fwd(p, **t), slra.residual_norm_bwd(p, **t, **d, workspace=w))
            assert slra.lib().slra_residual_norm_bwd(
                ctypes.byref(c), t["x"].data_ptr(), t["y"].data_ptr(), d["dx_out"].data_ptr(), d["dh"].data_ptr(),
                own["dx"].data_ptr(), own["dy"].data_ptr(), None, 0, torch.cuda.current_stream().cuda_stream) == slra.OK
        graphs.append((g, res))
    t["x"].mul_(0.5)
    d["dh"].mul_(2.0)
    for g, _ in graphs:
        g.replay()
    f, ref = slra.residual_norm_fwd(p, **t), slra.residual_norm_bwd(p, **t, **d)
    assert all(torch.equal(own[n], getattr(ref, n)) for n in names)
    for _, (gf, gb) in graphs:
        assert torch.equal(gf[0], f[0]) and torch.equal(gf[1], f[1])
        assert all(torch.equal(getattr(gb, n), getattr(ref, n)) for n in names)


# ------------------------------------------------------------------------------------------ qk rope
def rope_pairs(D, split=(0, 0, 0), schedule=slra.ROPE_PER_AXIS, theta=1e4):
    """[(axis, omega)] of the rotated pairs."""
    c = D // 2
    split = split if any(split) else (c - 2 * (c // 3), c // 3, c // 3)
    n, out = sum(split), []
    for ax in range(3):
        for m in range(split[ax]):
            out.append((ax, theta ** -(len(out) / n if schedule == slra.ROPE_SHARED else m / split[ax])))
    return out


def rope_inputs(B, L, hq, hk, D, x=BF, out=None, weights=FP, norm=slra.QK_NORM_HEAD, seed=0, **kw):
    g = torch.Generator(device="cuda").manual_seed(seed)
    p = slra.QkRope(B, L, hq, D, kv_heads=hk, norm=norm, **kw)
    t = {"q": rnd(g, (B, L, hq, D), x), "k": rnd(g, (B, L, hk, D), x) if hk else None, "wq": None, "wk": None}
    if norm != slra.QK_NORM_NONE and weights is not None:
        t["wq"] = rnd(g, ((hq if norm == slra.QK_NORM_TOKEN else 1) * D,), weights, 0.2, 1.0)
        if hk:
            t["wk"] = rnd(g, ((hk if norm == slra.QK_NORM_TOKEN else 1) * D,), weights, 0.2, 1.0)
    out = x if out is None else out
    d = {"dout_q": rnd(g, (B, L, hq, D), out, 0.1), "dout_k": rnd(g, (B, L, hk, D), out, 0.1) if hk else None}
    return p, t, d


def rope_reference(p, t, positions=None, d=None):
    """{name: (value, M)} in double."""
    B, L, D = p.batch, p.tokens, p.head_dim
    if positions is None:
        T, H, W = p.grid if p.grid is not None else (1, 1, L)
        n = torch.arange(p.first_token, p.first_token + L, device="cuda")
        positions = torch.stack([n // (H * W), n // W % H, n % W], 1)[None]
    pos = positions.double() + torch.tensor(p.pos_offset, device="cuda", dtype=torch.float64)
    cos, sin = torch.ones((pos.shape[0], L, 1, D // 2), device="cuda", dtype=torch.float64), None
    sin = torch.zeros_like(cos)
    if p.rotate:
        for j, (ax, omega) in enumerate(rope_pairs(D, p.rope_split, p.schedule, p.theta)):
            cos[:, :, 0, j], sin[:, :, 0, j] = (pos[..., ax] * omega).cos(), (pos[..., ax] * omega).sin()

    def pairs(v):
        return (v[..., :D // 2], v[..., D // 2:]) if p.pairing == slra.ROPE_HALVES else (v[..., 0::2], v[..., 1::2])

    def join(a, b):
        return torch.cat([a, b], -1) if p.pairing == slra.ROPE_HALVES else torch.stack([a, b], -1).flatten(-2)

    def turn(v, sgn):
        a, b = pairs(v)
        return join(a * cos - sgn * b * sin, sgn * a * sin + b * cos)

    def bound(v):
        a, b = pairs(v.abs())
        if not p.rotate:
            return v.abs()
        return join(a + b, a + b)

    dims = {slra.QK_NORM_NONE: None, slra.QK_NORM_HEAD: (3,), slra.QK_NORM_TOKEN: (2, 3)}[p.norm]
    out = {}
    for n in ("q", "k"):
        if t[n] is None:
            continue
        x = t[n].double()
        r = torch.rsqrt((x * x).mean(dims, keepdim=True) + p.eps) if dims else torch.ones_like(x)
        nrm = x * r
        w = torch.ones((), device="cuda", dtype=torch.float64) if t["w" + n] is None else t["w" + n].double().view(-1, D)
        if d is None:
            out["out_" + n] = (turn(nrm * w, 1.0), bound(nrm * w))
            continue
        g, Mg = turn(d["dout_" + n].double(), -1.0), bound(d["dout_" + n].double())
        if dims is None:
            out["d" + n] = (g, Mg)
            continue
        out["d" + n] = (r * (g * w - nrm * (g * w * nrm).mean(dims, keepdim=True)),
                        r * (Mg * w.abs() + nrm.abs() * (Mg * w.abs() * nrm.abs()).mean(dims, keepdim=True)))
        if t["w" + n] is not None:
            over = (0, 1) if p.norm == slra.QK_NORM_TOKEN else (0, 1, 2)
            out["dw" + n] = ((g * nrm).sum(over).flatten(), (Mg * nrm.abs()).sum(over).flatten())
    return out


def check_rope(p, t, d, positions=None):
    outs = slra.qk_rope_fwd(p, **t, positions=positions)
    ref = rope_reference(p, t, positions)
    for n, o in zip(("out_q", "out_k"), outs):
        assert (o is not None) == (n in ref)
        if o is not None:
            close(o, *ref[n], n)
    got = slra.qk_rope_bwd(p, t["q"], t["k"], **d, wq=t["wq"], wk=t["wk"], positions=positions)
    ref = rope_reference(p, t, positions, d)
    # a worker's own rows, and for a weight of all heads its heads
    rows = K_ROW + -(-p.batch * p.tokens // 148) + (0 if p.norm == slra.QK_NORM_TOKEN else p.heads + p.kv_heads)
    for n in ("dq", "dk", "dwq", "dwk"):
        g = getattr(got, n)
        assert (g is not None) == (n in ref), n
        if g is not None:
            close(g, *ref[n], n, K_ROW if n in ("dq", "dk") else rows)


NORMS = [slra.QK_NORM_NONE, slra.QK_NORM_HEAD, slra.QK_NORM_TOKEN]


@pytest.mark.parametrize("norm", NORMS)
@pytest.mark.parametrize("pairing", [slra.ROPE_INTERLEAVED, slra.ROPE_HALVES])
@pytest.mark.parametrize("B,L,hq,hk,D", [(1, 1, 1, 0, 64), (1, 1, 12, 12, 128), (2, 17, 2, 2, 64), (3, 50, 3, 1, 8),
                                         (1, 40, 5, 2, 96), (2, 33, 14, 2, 80), (1, 30, 24, 24, 128), (1, 21, 40, 40, 128),
                                         (1, 9, 7, 1, 256), (1, 700, 4, 4, 64), (1, 5, 64, 64, 128), (2, 2, 1, 1, 16),
                                         (1, 7, 1, 20, 64), (1, 13, 2, 9, 8), (2, 3, 33, 1, 128), (1, 9, 12, 7, 128),
                                         (300, 1, 3, 3, 64), (1, 6, 40, 21, 128), (1, 3, 1000, 700, 8)])
def test_rope_sizes(norm, pairing, B, L, hq, hk, D):
    p, t, d = rope_inputs(B, L, hq, hk, D, norm=norm, pairing=pairing, grid=(7, 9, 13), first_token=100, seed=L + hq)
    check_rope(p, t, d)


@pytest.mark.parametrize("norm", NORMS)
@pytest.mark.parametrize("hq,hk,D", [(55, 55, 96), (55, 7, 96), (64, 64, 80), (61, 1, 104), (31, 31, 248), (27, 3, 216), (9, 9, 72), (3, 1, 40), (1, 1, 24),
                                     (33, 8, 80), (12, 0, 96)])
def test_rope_heads_that_are_no_power_of_two(norm, hq, hk, D):
    """A thread for each vector of a head, or more where the block's threads do not divide into heads."""
    for pairing in (slra.ROPE_INTERLEAVED, slra.ROPE_HALVES):
        p, t, d = rope_inputs(1, 320, hq, hk, D, norm=norm, seed=hq + D, pairing=pairing, grid=(2, 16, 10), theta=1e4)
        check_rope(p, t, d)


@pytest.mark.parametrize("x,out", [(BF, BF), (HF, HF), (FP, FP), (BF, FP), (HF, FP)])
@pytest.mark.parametrize("norm", NORMS)
@pytest.mark.parametrize("pairing", [slra.ROPE_INTERLEAVED, slra.ROPE_HALVES])
def test_rope_types(x, out, norm, pairing):
    code = {BF: slra.DTYPE_BF16, HF: slra.DTYPE_F16, FP: slra.DTYPE_F32}[out]
    for weights in {FP, x, None}:
        p, t, d = rope_inputs(2, 19, 6, 2, 128, x, out, weights, norm, grid=(2, 4, 5), out_dtype=code, pairing=pairing)
        check_rope(p, t, d)


@pytest.mark.parametrize("kw", [dict(schedule=slra.ROPE_SHARED, theta=1e6), dict(rope_split=(10, 6, 16)),
                                dict(rope_split=(3, 0, 5)), dict(rope_split=(0, 0, 32)), dict(pos_offset=(5, -7, 1000)),
                                dict(rotate=False), dict(first_token=59), dict(theta=0.0)], ids=str)
def test_rope_options(kw):
    p, t, d = rope_inputs(2, 31, 3, 3, 64, FP, norm=slra.QK_NORM_TOKEN, **dict(dict(grid=(3, 5, 6)), **kw))
    if kw.get("theta") == 0.0:  # the default base
        ref = slra.QkRope(2, 31, 3, 64, kv_heads=3, norm=slra.QK_NORM_TOKEN, grid=(3, 5, 6))
        assert all(torch.equal(a, b) for a, b in zip(slra.qk_rope_fwd(p, **t), slra.qk_rope_fwd(ref, **t)))
        return
    check_rope(p, t, d)


@pytest.mark.parametrize("shared", [True, False])
@pytest.mark.parametrize("hq", [1, 20])
def test_rope_listed_positions(shared, hq):
    g = torch.Generator(device="cuda").manual_seed(4)
    p, t, d = rope_inputs(3, 45, hq, 1, 128, FP)
    pos = torch.randint(-40, 5000, (1 if shared else 3, 45, 3), generator=g, device="cuda", dtype=torch.int32)
    check_rope(p, t, d, pos)
    # the grid's own places, listed, give the grid's bits
    grid = slra.QkRope(3, 45, hq, 128, kv_heads=1, norm=slra.QK_NORM_HEAD, grid=(4, 5, 6), first_token=11)
    n = torch.arange(11, 56, device="cuda")
    listed = torch.stack([n // 30, n // 6 % 5, n % 6], 1)[None].int().contiguous()
    a, b = slra.qk_rope_fwd(grid, **t), slra.qk_rope_fwd(p, **t, positions=listed)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_rope_position_slices_and_single_weights():
    """Positions as a slice of a longer list; a weight for one side only; weights of another type."""
    g = torch.Generator(device="cuda").manual_seed(7)
    pos = torch.randint(0, 900, (3, 60, 3), generator=g, device="cuda", dtype=torch.int32)[:, 11:11 + 20]
    for side in ("wq", "wk"):
        for weights in (BF, HF, FP):
            for norm in (slra.QK_NORM_HEAD, slra.QK_NORM_TOKEN):
                p, t, d = rope_inputs(3, 20, 6, 4, 64, BF, weights=weights, norm=norm, seed=8)
                t[side] = None
                check_rope(p, t, d, pos)


def test_rope_far_positions():
    """Angles of far positions.  The product position * turns in double is off by two roundings (2^-53 each)
    of up to 2^31 / (2 pi) = 2^28.3 turns, 2 pi 2^-23.7 of angle: within three of the 64 fp32 roundings."""
    g = torch.Generator(device="cuda").manual_seed(5)
    p, t, d = rope_inputs(1, 64, 2, 2, 128, FP)
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (1, 64, 3), generator=g, device="cuda", dtype=torch.int64).int()
    pos[0, 0], pos[0, 1] = 2 ** 31 - 1, -2 ** 31
    check_rope(p, t, d, pos)


def test_rope_is_the_attentions():
    """The rotation of the attention's own preparation (fp16 q^ in the workspace), half an fp16 step apart
    from the fp32 result at most (plus the fp32 roundings of both)."""
    prob = slra.Problem(batch=1, heads=2, head_dim=128, T=3, H=6, W=8, block=64, keep_frac=0.5, rank=32)
    g = torch.Generator(device="cuda").manual_seed(6)
    q, k, v = (rnd(g, (1, 144, 2, 128), BF) for _ in range(3))
    ws = slra.select_blocks(prob, q, k, v)
    p = slra.QkRope(1, 144, 2, 128, kv_heads=2, grid=(3, 6, 8), out_dtype=slra.DTYPE_F32)
    for got, name in zip(slra.qk_rope_fwd(p, q, k), ("qh", "kh")):
        qh = slra.ws_view(prob, ws, name)[:, :144].permute(1, 0, 2)[None].double()
        a = got.double()
        assert ((qh - a).abs() <= 2.0 ** -11 * a.abs() + 16 * U32 * 8 + 2.0 ** -25).all()


def test_rope_fused_views_and_in_place():
    """q and k as views of one projection's output, rotated into themselves; gradients into a fused buffer."""
    B, L, hq, hk, D = 2, 23, 6, 2, 64
    p, t, d = rope_inputs(B, L, hq, hk, D, norm=slra.QK_NORM_TOKEN, grid=(2, 4, 3))
    ref = slra.qk_rope_fwd(p, **t)
    bwd = slra.qk_rope_bwd(p, t["q"], t["k"], **d, wq=t["wq"], wk=t["wk"])
    fused = torch.full((B, L, hq + 2 * hk, D), 3.0, dtype=BF, device="cuda")
    q, k, v = fused[:, :, :hq], fused[:, :, hq:hq + hk], fused[:, :, hq + hk:]
    q.copy_(t["q"]), k.copy_(t["k"])
    dfused = torch.full_like(fused, 5.0)
    dq, dk = dfused[:, :, :hq], dfused[:, :, hq:hq + hk]
    g = slra.qk_rope_bwd(p, q, k, **d, wq=t["wq"], wk=t["wk"], dq=dq, dk=dk)
    assert torch.equal(dq, bwd.dq) and torch.equal(dk, bwd.dk) and torch.equal(g.dwq, bwd.dwq)
    assert (dfused[:, :, hq + hk:] == 5).all()
    slra.qk_rope_fwd(p, q, k, t["wq"], t["wk"], out_q=q, out_k=k)
    assert torch.equal(q, ref[0]) and torch.equal(k, ref[1]) and (v == 3).all()
    # head-major tensors, gradients over the incoming ones
    hm = {n: t[n].permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for n in ("q", "k")}
    o = torch.empty((B, hq, L, D), dtype=BF, device="cuda").permute(0, 2, 1, 3)
    got = slra.qk_rope_fwd(p, hm["q"], hm["k"], t["wq"], t["wk"], out_q=o)
    assert got[0] is o and torch.equal(o, ref[0]) and torch.equal(got[1], ref[1])
    a, b = d["dout_q"].clone(), d["dout_k"].clone()
    slra.qk_rope_bwd(p, t["q"], t["k"], a, b, wq=t["wq"], wk=t["wk"], dq=a, dk=b)
    assert torch.equal(a, bwd.dq) and torch.equal(b, bwd.dk)


def test_rope_single_token_into_a_cache():
    """One new token a call, its key written to its place in a cache: the whole sequence's bits, and the
    cache's other places as they were."""
    B, L, hq, hk, D = 3, 10, 4, 2, 128
    p, t, _ = rope_inputs(B, L, hq, hk, D, grid=(5, 2, 2), norm=slra.QK_NORM_HEAD)
    ref = slra.qk_rope_fwd(p, **t)
    cache = torch.full((B, L + 3, hk, D), 9.0, dtype=BF, device="cuda")
    for n in range(L):
        one = slra.QkRope(B, 1, hq, D, kv_heads=hk, grid=(5, 2, 2), first_token=n, norm=slra.QK_NORM_HEAD)
        q, _ = slra.qk_rope_fwd(one, t["q"][:, n:n + 1], t["k"][:, n:n + 1], t["wq"], t["wk"], out_k=cache[:, n:n + 1])
        assert torch.equal(q, ref[0][:, n:n + 1])
        assert (cache[:, n + 1:] == 9).all()
    assert torch.equal(cache[:, :L], ref[1])


def test_rope_zero_rows_infinities_and_nan():
    p, t, _ = rope_inputs(1, 6, 2, 0, 64, norm=slra.QK_NORM_HEAD)
    ref, _ = slra.qk_rope_fwd(p, **t)
    t["q"][0, 1] = 0
    t["q"][0, 3, 0, 5] = float("nan")
    t["q"][0, 4, 1, 7] = float("inf")
    out, _ = slra.qk_rope_fwd(p, **t)
    assert not out[0, 1].any() and out[0, 3, 0].isnan().all() and out[0, 4, 1].isnan().any()
    for n, h in ((0, 0), (2, 1), (3, 1), (4, 0), (5, 0)):
        assert torch.equal(out[0, n, h], ref[0, n, h])


@pytest.mark.parametrize("norm", NORMS)
def test_rope_gradients_against_differences(norm):
    p, t, d = rope_inputs(1, 11, 3, 2, 16, FP, norm=norm, grid=(2, 3, 4))
    g = slra.qk_rope_bwd(p, t["q"], t["k"], **d, wq=t["wq"], wk=t["wk"])

    def loss(tt):
        r = rope_reference(p, tt)
        return float(sum((r["out_" + n][0] * d["dout_" + n].double()).sum() for n in ("q", "k")))

    gen = torch.Generator(device="cuda").manual_seed(2)
    for name in ("q", "k", "wq", "wk"):
        if t[name] is None:
            continue
        v = torch.randn(t[name].shape, generator=gen, device="cuda", dtype=torch.float64)
        e = 1e-4
        slope = (loss(dict(t, **{name: t[name].double() + e * v})) - loss(dict(t, **{name: t[name].double() - e * v}))) / (2 * e)
        terms = getattr(g, "d" + name).double() * v
        assert abs(float(terms.sum()) - slope) <= 1e-5 * float(terms.abs().sum()), name


@pytest.mark.parametrize("norm", [slra.QK_NORM_HEAD, slra.QK_NORM_TOKEN])
def test_rope_deterministic_streams_and_graphs(norm):
    import ctypes
    p, t, d = rope_inputs(1, 1500, 6, 2, 128, norm=norm, grid=(3, 20, 25))
    w = dict(wq=t["wq"], wk=t["wk"])
    ref, f = slra.qk_rope_bwd(p, t["q"], t["k"], **d, **w), slra.qk_rope_fwd(p, **t)
    names = ("dq", "dk", "dwq", "dwk")
    ws = ref.workspace
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other, fo = slra.qk_rope_bwd(p, t["q"], t["k"], **d, **w, stream=s), slra.qk_rope_fwd(p, **t, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    again = slra.qk_rope_bwd(p, t["q"], t["k"], **d, **w, workspace=ws)
    for n in names:
        assert torch.equal(getattr(other, n), getattr(ref, n)) and torch.equal(getattr(again, n), getattr(ref, n))
    assert torch.equal(fo[0], f[0]) and torch.equal(fo[1], f[1])
    c = slra._qk_rope_problem(p, t["q"], t["k"], t["wq"], t["wk"], None)[0]
    c.out_dtype = c.x_dtype
    own = {n: torch.empty_like(getattr(ref, n)) for n in names}
    c.dwq, c.dwk = own["dwq"].data_ptr(), own["dwk"].data_ptr()
    assert slra.lib().slra_qk_rope_bwd(ctypes.byref(c), t["q"].data_ptr(), t["k"].data_ptr(), d["dout_q"].data_ptr(),
                                       d["dout_k"].data_ptr(), own["dq"].data_ptr(), own["dk"].data_ptr(), None, 0,
                                       torch.cuda.current_stream().cuda_stream) == slra.OK
    assert all(torch.equal(own[n], getattr(ref, n)) for n in names)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gf, gb = slra.qk_rope_fwd(p, **t), slra.qk_rope_bwd(p, t["q"], t["k"], **d, **w, workspace=ws)
    t["q"].mul_(0.5)
    d["dout_k"].mul_(2.0)
    graph.replay()
    ref, f = slra.qk_rope_bwd(p, t["q"], t["k"], **d, **w), slra.qk_rope_fwd(p, **t)
    assert torch.equal(gf[0], f[0]) and torch.equal(gf[1], f[1])
    assert all(torch.equal(getattr(gb, n), getattr(ref, n)) for n in names)


# -------------------------------------------------------------------------------- refusals, together
def test_refusals_on_the_gpu():
    """What the documentation excludes is refused before anything is launched."""
    p, t, d = norm_inputs(1, 8, 64)
    with pytest.raises(slra.SlraError):  # x_out over y
        slra.residual_norm_fwd(p, **t, x_out=t["y"])
    with pytest.raises(slra.SlraError):  # rows shifted by one: overlap that is not the same rows
        buf = torch.zeros((1, 9, 64), dtype=BF, device="cuda")
        slra.residual_norm_fwd(p, buf[:, :8], t["y"], x_out=buf[:, 1:])
    with pytest.raises(slra.SlraError):
        slra.residual_norm_fwd(slra.ResidualNorm(1, 8, 64, residual_scale=0.5), t["x"])
    with pytest.raises(slra.SlraError):
        slra.residual_norm_fwd(slra.ResidualNorm(1, 8, 64, groups=3), t["x"], t["y"])
    with pytest.raises(ValueError):
        slra.residual_norm_fwd(p, t["x"].cpu(), t["y"])
    with pytest.raises(ValueError):  # an expanded row tensor
        slra.residual_norm_fwd(p, t["x"], t["y"][:, :1].expand(1, 8, 64))
    with pytest.raises(ValueError):
        slra.residual_norm_fwd(p, t["x"], t["y"], scale=t["scale"][:, :, :32])
    with pytest.raises(slra.SlraError):  # bf16 stream with fp16 blocks
        slra.residual_norm_fwd(p, t["x"], t["y"].to(HF))
    with pytest.raises(slra.SlraError):
        slra.residual_norm_bwd(p, **t, **d, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(slra.SlraError):  # channels above the limit
        big = torch.zeros((1, 1, 8200), dtype=BF, device="cuda")
        slra.residual_norm_fwd(slra.ResidualNorm(1, 1, 8200), big)
    with pytest.raises(slra.SlraError):  # misaligned rows
        odd = torch.zeros((1, 8, 68), dtype=BF, device="cuda")[:, :, :64]
        slra.residual_norm_fwd(p, odd, t["y"])
    p, t, d = rope_inputs(1, 8, 2, 2, 64, grid=(1, 2, 4))
    with pytest.raises(slra.SlraError):
        slra.qk_rope_fwd(slra.QkRope(1, 8, 2, 64, kv_heads=2, grid=(1, 2, 3)), t["q"], t["k"])
    with pytest.raises(slra.SlraError):
        slra.qk_rope_fwd(p, **t, out_q=t["k"])
    with pytest.raises(ValueError):
        slra.qk_rope_fwd(p, t["q"])
    with pytest.raises(ValueError):
        slra.qk_rope_fwd(p, **t, positions=torch.zeros((1, 8, 3), dtype=torch.int64, device="cuda"))
    with pytest.raises(slra.SlraError):
        slra.qk_rope_bwd(p, t["q"], t["k"], **d, wq=t["wq"], wk=t["wk"],
                         workspace=torch.empty(256, dtype=torch.uint8, device="cuda")[:128])


def test_block_half_with_the_attention():
    """The operators as a block uses them: norm of the stream, one QKV product, QK norm into the hybrid
    attention, gated residual and the next norm; then the chain backwards to the stream, the modulation
    rows and the QK weights.  Each stage is checked on the inputs it was given, so the tolerances are its
    own; the attention's stage is checked by its parity tests."""
    B, T, H, W, heads, D = 1, 3, 6, 8, 2, 128
    L, C = T * H * W, heads * D
    g = torch.Generator(device="cuda").manual_seed(21)
    x = rnd(g, (B, L, C), FP)
    mods = {n: rnd(g, (B, T, C), FP, 0.3) for n in ("scale0", "shift0", "gate", "scale1", "shift1")}
    wqkv, wo = rnd(g, (3 * C, C), BF, C ** -0.5), rnd(g, (C, C), BF, C ** -0.5)
    wq, wk = rnd(g, (C,), FP, 0.1, 1.0), rnd(g, (C,), FP, 0.1, 1.0)
    A = rnd(g, (D, 32), BF, D ** -0.5)
    first = slra.ResidualNorm(B, L, C, groups=T)
    qk = slra.QkRope(B, L, heads, D, kv_heads=heads, norm=slra.QK_NORM_TOKEN, rotate=False)
    attn = slra.Problem(batch=B, heads=heads, head_dim=D, T=T, H=H, W=W, block=64, keep_frac=0.5, rank=32)

    _, h0 = slra.residual_norm_fwd(first, x, scale=mods["scale0"], shift=mods["shift0"], h_dtype=BF)
    qkv = (h0 @ wqkv.t()).view(B, L, 3 * heads, D)
    q, k, v = qkv[:, :, :heads], qkv[:, :, heads:2 * heads], qkv[:, :, 2 * heads:]
    qn, kn = slra.qk_rope_fwd(qk, q, k, wq, wk)
    o, ws = slra.attn_fwd_train(attn, qn, kn, v, A)
    assert slra.device_status(ws) == slra.OK
    y = o.view(B, L, C).to(BF) @ wo.t()
    t = dict(x=x, y=y, gate=mods["gate"], scale=mods["scale1"], shift=mods["shift1"], weight=None, bias=None, post_weight=None)
    x1, h1 = slra.residual_norm_fwd(first, **t)
    ref = norm_reference(first, t)
    close(x1, *ref["x_out"], "x1"), close(h1, *ref["h"], "h1")
    ref = rope_reference(qk, dict(q=q, k=k, wq=wq, wk=wk))
    close(qn, *ref["out_q"], "qn"), close(kn, *ref["out_k"], "kn")

    d = dict(dh=rnd(g, (B, L, C), BF, 0.1), dx_out=rnd(g, (B, L, C), FP, 0.1))
    last = check_norm_backward(first, t, d)
    do = (last.dy @ wo).float().view(B, L, heads, D)
    dqn, dkn, dv, dA, _ = slra.attn_bwd_saved(attn, qn, kn, v, A, do, ws)
    assert slra.device_status(ws) == slra.OK
    dqkv = torch.empty_like(qkv)
    back = slra.qk_rope_bwd(qk, q, k, dqn, dkn, wq=wq, wk=wk, dq=dqkv[:, :, :heads], dk=dqkv[:, :, heads:2 * heads])
    dqkv[:, :, 2 * heads:] = dv
    ref = rope_reference(qk, dict(q=q, k=k, wq=wq, wk=wk), d=dict(dout_q=dqn, dout_k=dkn))
    for n in ("dq", "dk"):
        close(getattr(back, n), *ref[n], n)
    for n in ("dwq", "dwk"):
        close(getattr(back, n), *ref[n], n, K_ROW + 1)
    dh0 = (dqkv.view(B, L, 3 * C) @ wqkv)
    t0 = dict(x=x, y=None, gate=None, scale=mods["scale0"], shift=mods["shift0"], weight=None, bias=None, post_weight=None)
    check_norm_backward(first, t0, dict(dh=dh0, dx_out=last.dx))


def unrotated(D, split, pairing):
    """Mask [D] of the elements that a split leaves alone."""
    j = torch.arange(D, device="cuda")
    pair = j % (D // 2) if pairing == slra.ROPE_HALVES else j // 2
    return pair >= sum(split)


def same_bits(a, b):
    ints = {2: torch.int16, 4: torch.int32}[a.element_size()]
    return torch.equal(a.contiguous().view(ints), b.contiguous().view(ints))


@pytest.mark.parametrize("x,out", [(BF, BF), (HF, HF), (FP, FP), (BF, FP)])
@pytest.mark.parametrize("pairing", [slra.ROPE_INTERLEAVED, slra.ROPE_HALVES])
@pytest.mark.parametrize("D,split", [(64, (3, 0, 5)), (128, (1, 0, 0)), (40, (7, 6, 6)), (8, (0, 2, 0))])
def test_rope_pairs_that_are_not_rotated_pass_through(x, out, pairing, D, split):
    """Their bits arrive as they are, forward and backward: infinities, NaN and zeros of either sign, which a
    product with (1, 0) would spread to the pair's other element or lose."""
    code = {BF: slra.DTYPE_BF16, HF: slra.DTYPE_F16, FP: slra.DTYPE_F32}[out]
    for hq, hk in ((3, 1), (20, 20)):
        p, t, d = rope_inputs(2, 33, hq, hk, D, x, out, norm=slra.QK_NORM_NONE, pairing=pairing, rope_split=split, grid=(3, 4, 3),
                              out_dtype=code, seed=50)
        keep = unrotated(D, split, pairing)
        special = torch.tensor([float("inf"), -float("inf"), float("nan"), -0.0, 0.0], device="cuda")
        for v in (t["q"], t["k"], d["dout_q"], d["dout_k"]):
            at = (torch.rand(v.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(51)) < 0.2) & keep
            v[at] = special[torch.arange(int(at.sum()), device="cuda") % 5].to(v.dtype)
        clean = {n: None if v is None else torch.where(keep, torch.ones_like(v), v) for n, v in t.items()}
        cleand = {n: torch.where(keep, torch.ones_like(v), v) for n, v in d.items()}
        outs, ref = slra.qk_rope_fwd(p, **t), slra.qk_rope_fwd(p, **clean)
        got, gref = slra.qk_rope_bwd(p, t["q"], t["k"], **d), slra.qk_rope_bwd(p, clean["q"], clean["k"], **cleand)
        for o, r, v in ((outs[0], ref[0], t["q"]), (outs[1], ref[1], t["k"]), (got.dq, gref.dq, d["dout_q"]), (got.dk, gref.dk, d["dout_k"])):
            want = v.to(o.dtype)
            nan = want.isnan()
            assert torch.equal(o.isnan(), nan)
            assert same_bits(o.masked_fill(nan, 0)[..., keep], want.masked_fill(nan, 0)[..., keep])
            assert same_bits(o[..., ~keep], r[..., ~keep])  # the rotated ones never see them


@pytest.mark.parametrize("pairing", [slra.ROPE_INTERLEAVED, slra.ROPE_HALVES])
@pytest.mark.parametrize("x", [BF, HF, FP])
def test_rope_norm_alone_keeps_elements_apart(x, pairing):
    """Without a rotation an infinity makes its own element NaN (inf times a reciprocal of zero) and the others of
    its norm zero; in the gradient of the weights it stays in its own column."""
    for norm, hq in ((slra.QK_NORM_HEAD, 2), (slra.QK_NORM_TOKEN, 2), (slra.QK_NORM_HEAD, 30), (slra.QK_NORM_TOKEN, 30)):
        p, t, d = rope_inputs(1, 9, hq, 0, 64, x, norm=norm, rotate=False, pairing=pairing, seed=52)
        t["q"][0, 4, 1, 7] = float("inf")
        out, _ = slra.qk_rope_fwd(p, **t)
        hit = out[0, 4] if norm == slra.QK_NORM_TOKEN else out[0, 4, 1:2]
        at = 1 if norm == slra.QK_NORM_TOKEN else 0
        assert hit[at, 7].isnan() and int(hit.isnan().sum()) == 1 and int((hit == 0).sum()) == hit.numel() - 1
        assert int(out.isnan().sum()) == 1
        p, t, d = rope_inputs(1, 9, hq, 0, 64, x, norm=norm, rotate=False, pairing=pairing, seed=52)
        d["dout_q"][0, 4, 1, 7] = float("inf")
        g = slra.qk_rope_bwd(p, t["q"], None, d["dout_q"], wq=t["wq"])
        column = 64 + 7 if norm == slra.QK_NORM_TOKEN else 7
        assert g.dwq[column].isinf() and int(g.dwq.isfinite().sum()) == g.dwq.numel() - 1


@pytest.mark.parametrize("x,out", [(BF, BF), (HF, HF), (FP, FP), (BF, FP), (HF, FP)])
@pytest.mark.parametrize("norm", [slra.QK_NORM_HEAD, slra.QK_NORM_TOKEN])
@pytest.mark.parametrize("B,L,hq,hk,D", [(1, 1, 12, 12, 128), (2, 700, 12, 12, 128), (1, 900, 40, 40, 128), (3, 41, 24, 3, 80),
                                         (1, 77, 5, 0, 64)])
def test_rope_norm_alone(x, out, norm, B, L, hq, hk, D):
    """The QK norm as the attention wants it, gradients in fp32 as its backward writes them."""
    code = {BF: slra.DTYPE_BF16, HF: slra.DTYPE_F16, FP: slra.DTYPE_F32}[out]
    p, t, d = rope_inputs(B, L, hq, hk, D, x, out, x, norm, rotate=False, out_dtype=code, seed=53)
    check_rope(p, t, d)


def test_calls_from_several_host_threads_at_once():
    """Calls of one kernel at several sizes of its shared memory, from host threads of their own: none is refused,
    and every answer has its bits."""
    import ctypes
    import threading
    L = slra.lib()
    cases = []
    for C in (5120, 4096, 2560):
        p, t, d = norm_inputs(1, 1500, C, seed=C)
        ref = slra.residual_norm_bwd(p, **t, **d)
        f = slra.residual_norm_fwd(p, **t)
        c = slra._residual_norm_problem(p, t["x"], t["y"], d["dh"], *(t[n] for n in ("gate", "scale", "shift", "weight", "bias",
                                                                                     "post_weight")))[0]
        own, ob = [torch.empty_like(v) for v in f], [torch.empty_like(v) for v in (ref.dx, ref.dy)]
        a = [v.data_ptr() for v in (t["x"], t["y"], *own)]
        b = [v.data_ptr() for v in (t["x"], t["y"], d["dx_out"], d["dh"], *ob)]
        cases.append((lambda s, c=c, a=a: L.slra_residual_norm_fwd(ctypes.byref(c), *a, s), own, f, (t, c)))
        cases.append((lambda s, c=c, b=b: L.slra_residual_norm_bwd(ctypes.byref(c), *b, None, 0, s), ob, (ref.dx, ref.dy), (d, c)))
    for heads in (40, 32, 20):
        p, t, d = rope_inputs(1, 1500, heads, heads, 128, grid=(5, 20, 15), seed=heads)
        f, g = slra.qk_rope_fwd(p, **t), slra.qk_rope_bwd(p, t["q"], t["k"], **d, wq=t["wq"], wk=t["wk"])
        c = slra._qk_rope_problem(p, t["q"], t["k"], t["wq"], t["wk"], None)[0]
        c.out_dtype = c.x_dtype
        own, ob = [torch.empty_like(v) for v in f], [torch.empty_like(v) for v in (g.dq, g.dk)]
        a = [v.data_ptr() for v in (t["q"], t["k"], *own)]
        b = [v.data_ptr() for v in (t["q"], t["k"], d["dout_q"], d["dout_k"], *ob)]
        cases.append((lambda s, c=c, a=a: L.slra_qk_rope_fwd(ctypes.byref(c), *a, s), own, f, (t, c)))
        cases.append((lambda s, c=c, b=b: L.slra_qk_rope_bwd(ctypes.byref(c), *b, None, 0, s), ob, (g.dq, g.dk), (d, c)))
    torch.cuda.synchronize()
    streams, refused = [torch.cuda.Stream() for _ in cases], [0] * len(cases)
    start = threading.Barrier(len(cases))

    def work(i):
        call, s = cases[i][0], streams[i].cuda_stream
        start.wait()
        for _ in range(2000):
            refused[i] += call(s) != slra.OK

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert refused == [0] * len(cases)
    for _, got, ref, _ in cases:
        assert all(torch.equal(a, b) for a, b in zip(got, ref))


@pytest.mark.parametrize("order", ["token", "head"])
def test_rope_slices_of_one_buffer_over_a_batch(order):
    """q and k as slices of one [B, 3, ...] tensor, rotated in place, and gradients into slices of one: the samples of
    the slices interleave, their elements do not meet."""
    B, L, H, D = 3, 23, 4, 64
    p, t, d = rope_inputs(B, L, H, H, D, norm=slra.QK_NORM_HEAD, grid=(2, 4, 3), seed=54)
    ref, bwd = slra.qk_rope_fwd(p, **t), slra.qk_rope_bwd(p, t["q"], t["k"], **d, wq=t["wq"], wk=t["wk"])

    def slices(fill):
        if order == "token":
            buf = torch.full((B, 3, L, H, D), fill, dtype=BF, device="cuda")
            return buf, [buf[:, i] for i in range(3)]
        buf = torch.full((B, 3, H, L, D), fill, dtype=BF, device="cuda")
        return buf, [buf[:, i].transpose(1, 2) for i in range(3)]

    _, (q, k, v) = slices(3.0)
    q.copy_(t["q"]), k.copy_(t["k"])
    _, (dq, dk, dv) = slices(5.0)
    slra.qk_rope_bwd(p, q, k, **d, wq=t["wq"], wk=t["wk"], dq=dq, dk=dk)
    assert torch.equal(dq, bwd.dq) and torch.equal(dk, bwd.dk) and (dv == 5).all()
    slra.qk_rope_fwd(p, q, k, t["wq"], t["wk"], out_q=q, out_k=k)
    assert torch.equal(q, ref[0]) and torch.equal(k, ref[1]) and (v == 3).all()


def test_norm_slices_of_one_buffer_over_a_batch():
    """x, y, x_out and h as slices of one [B, 4, L, C] tensor, gradients into slices of one."""
    B, L, C = 3, 29, 320
    p, t, d = norm_inputs(B, L, C, seed=55)
    ref, bwd = slra.residual_norm_fwd(p, **t), slra.residual_norm_bwd(p, **t, **d)
    buf = torch.full((B, 4, L, C), 3.0, dtype=BF, device="cuda")
    x, y, x_out, h = (buf[:, i] for i in range(4))
    x.copy_(t["x"]), y.copy_(t["y"])
    s = dict(t, x=x, y=y)
    slra.residual_norm_fwd(p, **s, x_out=x_out, h=h)
    assert torch.equal(x_out, ref[0]) and torch.equal(h, ref[1]) and torch.equal(x, t["x"]) and torch.equal(y, t["y"])
    x_out.copy_(d["dx_out"]), h.copy_(d["dh"])
    out = torch.full((B, 3, L, C), 5.0, dtype=BF, device="cuda")
    slra.residual_norm_bwd(p, **s, dx_out=x_out, dh=h, dx=out[:, 2], dy=out[:, 0])
    assert torch.equal(out[:, 2], bwd.dx) and torch.equal(out[:, 0], bwd.dy) and (out[:, 1] == 5).all()
    slra.residual_norm_bwd(p, **s, dx_out=x_out, dh=h, dx=x_out, dy=h)
    assert torch.equal(x_out, bwd.dx) and torch.equal(h, bwd.dy)


@pytest.mark.parametrize("schedule", [slra.ROPE_PER_AXIS, slra.ROPE_SHARED])
def test_rope_angles_of_far_positions(schedule):
    """Positions and offsets of up to 2^31 each, against angles reduced in 60 digits (a product in double is off by
    more than the kernel here).  An angle is p times turns, turns the integer part of 2^64 omega / 2 pi: at most 2.5
    units off with the long double powers, so 2.5 2^-32 turns at |p| = 2^32; 2^-32 turns for the lower half that is
    dropped; the fraction's rounding to fp32, 2^-25 half turns: 1.7 2^-24 in all.  cos and sin: 2 2^-24; a product
    and an fma of it: 2 2^-24.  Within 6 roundings of |a| + |b|."""
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    two_pi = Decimal("6.28318530717958647692528676655900576839433879875021164194989")
    L, D, offset = 48, 128, (2 ** 31, -2 ** 31, 12345)
    p, t, d = rope_inputs(1, L, 2, 1, D, FP, norm=slra.QK_NORM_NONE, schedule=schedule, pos_offset=offset, seed=60)
    g = torch.Generator(device="cuda").manual_seed(61)
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (1, L, 3), generator=g, device="cuda", dtype=torch.int64).int()
    pos[0, 0], pos[0, 1], pos[0, 2] = 2 ** 31 - 1, -2 ** 31, 0
    c = D // 2
    split = (c - 2 * (c // 3), c // 3, c // 3)
    angle = []
    for row in pos[0].tolist():
        for ax in range(3):
            for m in range(split[ax]):
                power = Decimal(sum(split[:ax]) + m) / c if schedule == slra.ROPE_SHARED else Decimal(m) / split[ax]
                turns = (row[ax] + offset[ax]) * (-power * Decimal(10000).ln()).exp() / two_pi
                angle.append(float((turns - turns.to_integral_value()) * two_pi))
    angle = torch.tensor(angle, dtype=torch.float64, device="cuda").view(1, L, 1, c)
    outs = slra.qk_rope_fwd(p, t["q"], t["k"], positions=pos)
    back = slra.qk_rope_bwd(p, t["q"], t["k"], **d, positions=pos)
    for got, v, sgn in ((outs[0], t["q"], 1), (outs[1], t["k"], 1), (back.dq, d["dout_q"], -1), (back.dk, d["dout_k"], -1)):
        a, b = v.double()[..., 0::2], v.double()[..., 1::2]
        cos, sin = angle.cos(), sgn * angle.sin()
        ref = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        M = (a.abs() + b.abs()).repeat_interleave(2, dim=-1)
        close(got, ref, M, "far positions", 6)
