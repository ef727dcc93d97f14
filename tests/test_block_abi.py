"""Host-side checks of the operators around the attention (no GPU needed): defaults, validation of
problems and arguments, workspace sizes.  Pointers are never dereferenced by the host."""
import ctypes

import pytest

from sparse_rank_hybrid_b200 import build as B
from sparse_rank_hybrid_b200 import slra

BASE = 1 << 40  # made-up device addresses, 16 MiB apart


@pytest.fixture(scope="module", autouse=True)
def built():
    import torch
    B.build()
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: on a machine without a GPU only")


def at(i):
    return BASE + (i << 24)


def norm_problem(**kw):
    c = slra._ResidualNorm()
    assert slra.lib().slra_residual_norm_init(ctypes.byref(c), 2, 24, 64) == slra.OK
    for n, v in kw.items():
        if isinstance(v, tuple):
            getattr(c, n)[:] = v
        else:
            setattr(c, n, v)
    return c


def norm_fwd(c, x=at(0), y=at(1), x_out=at(2), h=at(3)):
    return slra.lib().slra_residual_norm_fwd(ctypes.byref(c), x, y, x_out, h, None)


def norm_bwd(c, x=at(0), y=at(1), dx_out=at(2), dh=at(3), dx=at(4), dy=at(5), ws=at(6), n=1 << 24):
    return slra.lib().slra_residual_norm_bwd(ctypes.byref(c), x, y, dx_out, dh, dx, dy, ws, n, None)


def test_norm_defaults_reach_the_device_check():
    c = norm_problem()
    assert (c.groups, c.norm, c.post_norm, c.stream_dtype, c.mod_dtype) == (1, slra.NORM_LAYER, slra.NORM_NONE,
                                                                             slra.DTYPE_BF16, slra.DTYPE_F32)
    assert tuple(c.gate_strides) == (-1, -1) and c.residual_scale == 1.0
    assert norm_fwd(c) == slra.ERR_NO_DEVICE and norm_bwd(c) == slra.ERR_NO_DEVICE
    assert slra.lib().slra_residual_norm_init(None, 1, 1, 8) == slra.ERR_INVALID_ARG
    assert norm_fwd(norm_problem(), y=None, x_out=None) == slra.ERR_NO_DEVICE
    assert norm_fwd(norm_problem(norm=slra.NORM_NONE), h=None) == slra.ERR_NO_DEVICE


@pytest.mark.parametrize("kw,status", [
    (dict(batch=0), slra.ERR_INVALID_ARG), (dict(tokens=0), slra.ERR_INVALID_ARG),
    (dict(channels=0), slra.ERR_INVALID_ARG), (dict(groups=0), slra.ERR_INVALID_ARG),
    (dict(groups=5), slra.ERR_INVALID_ARG), (dict(batch=1 << 16, tokens=1 << 16), slra.ERR_INVALID_ARG),
    (dict(channels=60), slra.ERR_UNSUPPORTED), (dict(channels=8200), slra.ERR_UNSUPPORTED),
    (dict(norm=3), slra.ERR_INVALID_ARG), (dict(post_norm=slra.NORM_LAYER), slra.ERR_INVALID_ARG),
    (dict(stream_dtype=3), slra.ERR_INVALID_ARG), (dict(mod_dtype=-1), slra.ERR_INVALID_ARG),
    (dict(block_dtype=slra.DTYPE_F16), slra.ERR_UNSUPPORTED),
    (dict(stream_dtype=slra.DTYPE_F16, block_dtype=slra.DTYPE_F32), slra.ERR_UNSUPPORTED),
    (dict(eps=0.0), slra.ERR_INVALID_ARG), (dict(eps=float("nan")), slra.ERR_INVALID_ARG),
    (dict(post_eps=-1.0), slra.ERR_INVALID_ARG), (dict(residual_scale=float("inf")), slra.ERR_INVALID_ARG),
    (dict(norm=slra.NORM_NONE, scale=at(8)), slra.ERR_INVALID_ARG),
    (dict(norm=slra.NORM_RMS, bias=at(8)), slra.ERR_INVALID_ARG), (dict(post_weight=at(8)), slra.ERR_INVALID_ARG),
    (dict(dgate=at(8)), slra.ERR_INVALID_ARG), (dict(dweight=at(8)), slra.ERR_INVALID_ARG),
    (dict(scale=at(8) + 8), slra.ERR_ALIGNMENT), (dict(scale=at(8), dscale=at(9) + 4), slra.ERR_ALIGNMENT),
    (dict(x_strides=(2048, 68)), slra.ERR_INVALID_ARG), (dict(x_strides=(2048, 0)), slra.ERR_INVALID_ARG),
    (dict(scale=at(8), scale_strides=(-2, 0)), slra.ERR_INVALID_ARG),
    (dict(scale=at(8), scale_strides=(2, 0)), slra.ERR_INVALID_ARG),
    (dict(scale=at(8), scale_strides=(0, 0)), slra.ERR_NO_DEVICE),
    (dict(x_strides=(4096, 72)), slra.ERR_NO_DEVICE),
])
def test_norm_problem_validation(kw, status):
    c = norm_problem(**kw)
    assert norm_bwd(c) == status
    n = slra.lib().slra_residual_norm_bwd_workspace_bytes(ctypes.byref(c))
    assert (n > 0) == (status == slra.ERR_NO_DEVICE)


def test_norm_argument_validation():
    INV, DEV = slra.ERR_INVALID_ARG, slra.ERR_NO_DEVICE
    c = norm_problem()
    assert norm_fwd(c, x=None) == INV and norm_fwd(c, h=None) == INV and norm_fwd(c, x_out=None) == INV
    assert norm_fwd(c, y=None) == INV                        # x_out without y
    assert norm_fwd(c, x=at(0) + 8) == slra.ERR_ALIGNMENT
    assert norm_fwd(c, x_out=at(0)) == DEV and norm_fwd(c, h=at(1)) == DEV   # in place
    assert norm_fwd(c, x_out=at(1)) == INV and norm_fwd(c, h=at(0)) == INV and norm_fwd(c, h=at(2)) == INV
    assert norm_fwd(c, x_out=at(0) + 16) == INV
    assert norm_fwd(norm_problem(scale=at(3) + 64)) == INV   # h over scale
    assert norm_fwd(norm_problem(gate=at(8)), y=None, x_out=None) == INV
    assert norm_fwd(norm_problem(residual_scale=0.5), y=None, x_out=None) == INV
    assert norm_fwd(norm_problem(post_norm=slra.NORM_RMS), y=None, x_out=None) == INV
    assert norm_fwd(norm_problem(norm=slra.NORM_NONE), y=None, x_out=None, h=None) == INV
    assert norm_fwd(norm_problem(x_out_strides=(24 * 64, 32))) == INV  # output rows overlap
    # two views of one buffer, rows interleaved: no overlap unless their columns do
    i = dict(x_strides=(24 * 128, 128), x_out_strides=(24 * 128, 128))
    assert norm_fwd(norm_problem(**i), x=at(0), x_out=at(0) + 128) == DEV
    assert norm_fwd(norm_problem(**i), x=at(0), x_out=at(0) + 112) == INV
    assert norm_bwd(c, dx_out=None) == DEV and norm_bwd(c, dh=None) == INV and norm_bwd(c, dx=None) == INV
    assert norm_bwd(c, dx=at(2)) == DEV and norm_bwd(c, dy=at(3)) == DEV     # over dx_out, over dh
    assert norm_bwd(c, dx=at(0)) == INV and norm_bwd(c, dy=at(4)) == INV and norm_bwd(c, dy=at(1)) == INV
    assert norm_bwd(c, ws=at(0)) == INV
    v = norm_problem(gate=at(8), dgate=at(9), scale=at(10), dscale=at(11), weight=at(12), dweight=at(13))
    need = slra.lib().slra_residual_norm_bwd_workspace_bytes(ctypes.byref(v))
    assert norm_bwd(v) == DEV and norm_bwd(v, ws=None, n=0) == DEV
    assert norm_bwd(v, n=need - 1) == slra.ERR_WORKSPACE and norm_bwd(v, ws=at(6) + 16) == slra.ERR_WORKSPACE
    v.dscale = at(9)
    assert norm_bwd(v) == INV                                # two gradients in one place
    v.dscale = at(10)
    assert norm_bwd(v) == INV                                # a gradient over its vector


def rope_problem(**kw):
    c = slra._QkRope()
    assert slra.lib().slra_qk_rope_init(ctypes.byref(c), 2, 24, 4, 64) == slra.OK
    for n, v in dict(dict(kv_heads=2), **kw).items():
        if isinstance(v, tuple):
            getattr(c, n)[:] = v
        else:
            setattr(c, n, v)
    return c


def rope_fwd(c, q=at(0), k=at(1), oq=at(2), ok=at(3)):
    return slra.lib().slra_qk_rope_fwd(ctypes.byref(c), q, k, oq, ok, None)


def rope_bwd(c, q=at(0), k=at(1), gq=at(2), gk=at(3), dq=at(4), dk=at(5), ws=at(6), n=1 << 24):
    return slra.lib().slra_qk_rope_bwd(ctypes.byref(c), q, k, gq, gk, dq, dk, ws, n, None)


HEAD, TOKEN = slra.QK_NORM_HEAD, slra.QK_NORM_TOKEN


@pytest.mark.parametrize("kw,status", [
    (dict(), slra.ERR_NO_DEVICE), (dict(batch=0), slra.ERR_INVALID_ARG), (dict(heads=0), slra.ERR_INVALID_ARG),
    (dict(kv_heads=-1), slra.ERR_INVALID_ARG), (dict(head_dim=60), slra.ERR_UNSUPPORTED),
    (dict(head_dim=264), slra.ERR_UNSUPPORTED), (dict(heads=129), slra.ERR_UNSUPPORTED), (dict(kv_heads=129), slra.ERR_UNSUPPORTED),
    (dict(heads=128, kv_heads=128), slra.ERR_NO_DEVICE),
    (dict(heads=1 << 40), slra.ERR_UNSUPPORTED),
    (dict(batch=1 << 16, tokens=1 << 16), slra.ERR_INVALID_ARG), (dict(T=0), slra.ERR_INVALID_ARG),
    (dict(W=23), slra.ERR_INVALID_ARG), (dict(first_token=1), slra.ERR_INVALID_ARG),
    (dict(first_token=1, T=2), slra.ERR_NO_DEVICE), (dict(first_token=-1, T=2), slra.ERR_INVALID_ARG),
    (dict(W=1, positions=at(8)), slra.ERR_NO_DEVICE), (dict(positions=at(8) + 2), slra.ERR_ALIGNMENT),
    (dict(positions=at(8), positions_stride=71), slra.ERR_INVALID_ARG),
    (dict(positions=at(8), positions_stride=72), slra.ERR_NO_DEVICE), (dict(W=0, rotate=0, norm=HEAD), slra.ERR_NO_DEVICE),
    (dict(rotate=0), slra.ERR_INVALID_ARG),
    (dict(pos_offset=(0, (1 << 31) + 1, 0)), slra.ERR_INVALID_ARG), (dict(theta=float("nan")), slra.ERR_INVALID_ARG),
    (dict(theta=-1.0), slra.ERR_INVALID_ARG), (dict(theta=0.5), slra.ERR_INVALID_ARG),
    (dict(T=1 << 16, H=1 << 8, W=1 << 7), slra.ERR_INVALID_ARG), (dict(theta=1.0), slra.ERR_NO_DEVICE),
    (dict(q_strides=(1 << 35, 64, 1 << 31)), slra.ERR_UNSUPPORTED), (dict(rope_split=(20, 10, 3)), slra.ERR_INVALID_ARG),
    (dict(rope_split=(-1, 10, 3)), slra.ERR_INVALID_ARG), (dict(rope_split=(10, 10, 3)), slra.ERR_NO_DEVICE),
    (dict(norm=3), slra.ERR_INVALID_ARG), (dict(rotate=2), slra.ERR_INVALID_ARG), (dict(pairing=2), slra.ERR_INVALID_ARG),
    (dict(schedule=-1), slra.ERR_INVALID_ARG), (dict(x_dtype=3), slra.ERR_INVALID_ARG),
    (dict(x_dtype=slra.DTYPE_F32), slra.ERR_UNSUPPORTED), (dict(out_dtype=slra.DTYPE_F16), slra.ERR_UNSUPPORTED),
    (dict(out_dtype=slra.DTYPE_F32), slra.ERR_NO_DEVICE), (dict(eps=0.0, norm=HEAD), slra.ERR_INVALID_ARG),
    (dict(wq=at(8)), slra.ERR_INVALID_ARG), (dict(norm=HEAD, wq=at(8)), slra.ERR_NO_DEVICE),
    (dict(norm=HEAD, wq=at(8) + 8), slra.ERR_ALIGNMENT), (dict(norm=HEAD, dwq=at(8)), slra.ERR_INVALID_ARG),
    (dict(norm=HEAD, wq=at(8), dwq=at(9), wk=at(10), dwk=at(11)), slra.ERR_NO_DEVICE),
    (dict(norm=TOKEN, wq=at(8), dwq=at(9), wk=at(10), dwk=at(9)), slra.ERR_INVALID_ARG),
    (dict(q_strides=(24 * 256, 256, 60)), slra.ERR_INVALID_ARG), (dict(q_strides=(24 * 512, 512, 64)), slra.ERR_NO_DEVICE),
    (dict(dq_strides=(24 * 256, 256, 32)), slra.ERR_INVALID_ARG),  # rows of the gradient overlap
])
def test_rope_problem_validation(kw, status):
    assert rope_bwd(rope_problem(**kw)) == status


def test_rope_argument_validation():
    INV, DEV = slra.ERR_INVALID_ARG, slra.ERR_NO_DEVICE
    assert slra.lib().slra_qk_rope_init(None, 1, 1, 1, 64) == INV
    c = rope_problem()
    assert rope_fwd(c) == DEV and rope_fwd(c, q=None) == INV and rope_fwd(c, k=None) == INV and rope_fwd(c, ok=None) == INV
    assert rope_fwd(rope_problem(kv_heads=0), k=None, ok=None) == DEV and rope_fwd(rope_problem(kv_heads=0)) == INV
    assert rope_fwd(c, q=at(0) + 8) == slra.ERR_ALIGNMENT
    assert rope_fwd(c, oq=at(0), ok=at(1)) == DEV and rope_fwd(c, oq=at(1)) == INV and rope_fwd(c, ok=at(2)) == INV
    assert rope_fwd(c, oq=at(0) + 16) == INV
    # fused [q | k | v] rows, in place
    f = dict(zip(("q_strides", "k_strides", "out_q_strides", "out_k_strides"), [(24 * 512, 512, 64)] * 4))
    assert rope_fwd(rope_problem(**f), at(0), at(0) + 512, at(0), at(0) + 512) == DEV
    assert rope_fwd(rope_problem(**f), at(0), at(0) + 512, at(0) + 256, at(0) + 768) == INV
    # q at another stride of heads over the same bytes is not in place
    assert rope_fwd(rope_problem(heads=2, q_strides=(24 * 512, 512, 128), out_q_strides=(24 * 512, 512, 192)),
                    oq=at(0)) == INV
    # fp32 results over bf16 inputs are not in place
    assert rope_fwd(rope_problem(out_dtype=slra.DTYPE_F32), oq=at(0)) == INV
    assert rope_bwd(c, q=None, k=None) == DEV                # no norm: q and k are not read
    h = rope_problem(norm=HEAD, wq=at(8), dwq=at(9))
    assert rope_bwd(h) == DEV and rope_bwd(h, q=None) == INV and rope_bwd(h, k=None) == INV
    assert rope_bwd(h, dq=at(2), dk=at(3)) == DEV and rope_bwd(h, dq=at(0)) == INV and rope_bwd(h, dq=at(9)) == INV
    need = slra.lib().slra_qk_rope_bwd_workspace_bytes(ctypes.byref(h))
    assert rope_bwd(h, n=need - 1) == slra.ERR_WORKSPACE and rope_bwd(h, ws=None, n=0) == DEV
    assert rope_bwd(h, ws=at(0)) == INV and rope_bwd(rope_problem(positions=at(4) + 64, W=1)) == INV


def test_views_of_one_buffer_over_a_batch():
    """Slices of one buffer whose samples interleave do not meet; a row further they do."""
    INV, DEV = slra.ERR_INVALID_ARG, slra.ERR_NO_DEVICE
    B, L, H, D = 2, 24, 4, 64
    one = L * H * D  # elements of a sample's slice
    for token, head in ((H * D, D), (D, L * D)):  # [B, 3, L, H, D] and [B, 3, H, L, D]
        st = (3 * one, token, head)
        f = dict(kv_heads=4, **{n + "_strides": st for n in ("q", "k", "out_q", "out_k", "dq", "dk")})
        q, k, v = at(0), at(0) + 2 * one, at(0) + 4 * one
        assert rope_fwd(rope_problem(**f), q, k, q, k) == DEV and rope_fwd(rope_problem(**f), q, k, v, at(1)) == DEV
        assert rope_fwd(rope_problem(**f), q, k, q, k - 2 * D) == INV and rope_fwd(rope_problem(**f), q, k, at(1), v + 2 * D) == INV
        n = dict(f, norm=HEAD)
        assert rope_bwd(rope_problem(**n), at(0), at(0) + 2 * one, at(1), at(1) + 2 * one, at(2), at(2) + 2 * one) == DEV
        assert rope_bwd(rope_problem(**n), at(0), at(0) + 2 * one, at(1), at(1) + 2 * one, at(2), at(2) + 2 * one - 16) == INV
    one = 24 * 64
    s = {n + "_strides": (4 * one, 64) for n in ("x", "y", "x_out", "h")}
    slices = [at(0) + 2 * one * i for i in range(4)]
    assert norm_fwd(norm_problem(**s), *slices) == DEV and norm_fwd(norm_problem(**s), *slices[::-1]) == DEV
    assert norm_fwd(norm_problem(**s), *slices[:3], slices[3] + 16) == INV
    # a stride that a single sample never takes is nothing to compare
    assert norm_fwd(norm_problem(batch=1, x_strides=(8, 64)), x_out=at(0)) == DEV


def test_regions_against_every_piece():
    """The check of overlaps against the sets of pieces: never passes an overlap, and refuses views of the same
    strides only for one."""
    import random
    rng = random.Random(1)
    INV, DEV = slra.ERR_INVALID_ARG, slra.ERR_NO_DEVICE
    counts = {INV: 0, DEV: 0}
    for _ in range(4000):
        B, L, H = rng.randint(1, 3), rng.randint(1, 4), rng.randint(1, 4)
        def strides():
            dims, span, st = [(0, B), (1, L), (2, H)], 8, [8, 8, 8]
            rng.shuffle(dims)
            for i, n in dims:
                st[i] = span + 8 * rng.choice([0, 0, 0, 1, 2, 5, 12])
                span += st[i] * (n - 1)
            return tuple(st)
        a = strides()
        b = a if rng.random() < 0.7 else strides()
        d = 8 * rng.randint(-30, 30)
        def pieces(st, off):
            return {off + i * st[0] + j * st[1] + k * st[2] for i in range(B) for j in range(L) for k in range(H)}
        meet = bool(pieces(a, 0) & pieces(b, d))
        c = rope_problem(batch=B, tokens=L, W=L, heads=H, kv_heads=0, head_dim=8, q_strides=a, out_q_strides=b)
        got = rope_fwd(c, at(1), None, at(1) + 2 * d, None)
        in_place = d == 0 and all(x == y or n == 1 for x, y, n in zip(a, b, (B, L, H)))
        counts[got] += 1
        if meet and not in_place:
            assert got == INV, (B, L, H, a, b, d)
        elif a == b or in_place:
            assert got == DEV, (B, L, H, a, b, d)
    assert min(counts.values()) > 500


def test_head_strides_count_each_side():
    """A head-major cache of 2^20 tokens: the limit on a token's reach is that of the tensor's own heads."""
    far = 1 << 26  # 2^20 tokens of 64 elements
    k = dict(heads=64, kv_heads=8, k_strides=(far * 8, 64, far), out_k_strides=(far * 8, 64, far), dk_strides=(far * 8, 64, far))
    c = rope_problem(**k)
    assert rope_fwd(c, k=at(0) + (1 << 36), ok=at(0) + (1 << 37)) == slra.ERR_NO_DEVICE
    assert rope_bwd(c, k=at(0) + (1 << 36), gk=at(0) + (1 << 37), dk=at(0) + (1 << 38)) == slra.ERR_NO_DEVICE
    assert rope_fwd(rope_problem(**dict(k, kv_heads=33)), k=at(0) + (1 << 36), ok=at(0) + (1 << 37)) == slra.ERR_UNSUPPORTED
    q = dict(kv_heads=64, heads=8, q_strides=(far * 8, 64, far), out_q_strides=(far * 8, 64, far))
    assert rope_fwd(rope_problem(**q), q=at(0) + (1 << 36), oq=at(0) + (1 << 37)) == slra.ERR_NO_DEVICE


def test_workspaces_hold_a_bounded_number_of_partial_sums():
    """The partial sums grow with the workers, which are bounded, not with the tokens."""
    L = slra.lib()
    sizes = []
    for tokens in (1, 1000, 75600, 1 << 24):
        c = norm_problem(batch=1, tokens=tokens, channels=5120, gate=at(8), dgate=at(9))
        sizes.append(L.slra_residual_norm_bwd_workspace_bytes(ctypes.byref(c)))
        r = rope_problem(batch=1, tokens=tokens, W=tokens, norm=TOKEN, wq=at(8), dwq=at(9), heads=40, kv_heads=40,
                         head_dim=128)
        assert 0 < L.slra_qk_rope_bwd_workspace_bytes(ctypes.byref(r)) < 1 << 26
    assert sizes == sorted(sizes) and sizes[-1] == sizes[-2] < 1 << 26


def test_binding_checks_its_tensors():
    import torch
    x = torch.zeros((1, 4, 64))
    with pytest.raises(ValueError):
        slra.residual_norm_fwd(slra.ResidualNorm(1, 4, 64), x)
    with pytest.raises(ValueError):
        slra.qk_rope_fwd(slra.QkRope(1, 4, 1, 64), x.view(1, 4, 1, 64))
    with pytest.raises(ValueError):
        slra.residual_norm_fwd(slra.ResidualNorm(1, 4, 64), x.double())


@pytest.mark.parametrize("t,strides", [
    ("contiguous", (0, 0)), ("wide", (4 * 72, 72)), ("one sample", (8, 72)), ("one token", (72, 8)),
    ("expanded", None), ("expanded whole", None), ("last dimension", None), ("shape", None), ("type", None)])
def test_binding_strides(t, strides):
    """The binding's strides: zeros for a contiguous tensor only, never for an expanded one (the struct's
    zeros would read it as contiguous)."""
    import torch
    x = {"contiguous": torch.zeros(2, 4, 64), "wide": torch.zeros(2, 4, 72)[:, :, :64],
         "one sample": torch.zeros(1, 4, 72)[:, :, :64], "one token": torch.zeros(2, 1, 72)[:, :, :64],
         "expanded": torch.zeros(2, 1, 64).expand(2, 4, 64), "expanded whole": torch.zeros(64).expand(2, 4, 64),
         "last dimension": torch.zeros(2, 64, 4).transpose(1, 2), "shape": torch.zeros(2, 4, 72),
         "type": torch.zeros(2, 4, 64, dtype=torch.float64)}[t]
    shape = {"one sample": (1, 4, 64), "one token": (2, 1, 64)}.get(t, (2, 4, 64))
    c = slra._ResidualNorm()
    if strides is None:
        with pytest.raises(ValueError):
            slra._rows(c, "x", x, shape, torch.float32, x.device, "x_strides")
    else:
        assert slra._rows(c, "x", x, shape, torch.float32, x.device, "x_strides") == x.data_ptr()
        assert tuple(c.x_strides) == strides


def test_binding_refuses_another_type_of_h():
    """h has y's type: another one was given y's without a word."""
    import torch
    p, x, y = slra.ResidualNorm(1, 4, 64), torch.zeros((1, 4, 64)), torch.zeros((1, 4, 64), dtype=torch.bfloat16)
    for kw in (dict(y=y, h_dtype=torch.float32), dict(h=y, h_dtype=torch.float32), dict(h_dtype=torch.float64),
               dict(y=y, h=y, h_dtype=torch.float16)):
        with pytest.raises(ValueError, match="h_dtype"):
            slra.residual_norm_fwd(p, x, **kw)
    with pytest.raises(ValueError, match="CUDA"):  # the type itself is right
        slra.residual_norm_fwd(p, x, y=y, h_dtype=torch.bfloat16)


def test_binding_takes_lists_for_tuples():
    """A problem with lists gives the struct of one with tuples."""
    import torch
    q = torch.zeros((1, 24, 2, 64))
    kw = dict(grid=[2, 3, 4], pos_offset=[1, 2, 3], rope_split=[8, 8, 8])
    one = slra._qk_rope_problem(slra.QkRope(1, 24, 2, 64, **kw), q, None, None, None, None)[0]
    two = slra._qk_rope_problem(slra.QkRope(1, 24, 2, 64, **{n: tuple(v) for n, v in kw.items()}), q, None, None, None, None)[0]
    assert bytes(one) == bytes(two) and (one.T, one.H, one.W) == (2, 3, 4)


def test_binding_refuses_an_unknown_type_of_outputs():
    import torch
    q = torch.zeros((1, 24, 2, 64))
    for code in (7, torch.float32):
        with pytest.raises(ValueError, match="out_dtype"):
            slra.qk_rope_fwd(slra.QkRope(1, 24, 2, 64, out_dtype=code), q)


def test_binding_names_what_an_older_library_lacks(tmp_path, monkeypatch):
    """A library of the same ABI number from before functions were added."""
    import subprocess
    older = [n for n in slra.EXPORTS if not n.startswith(("slra_residual_norm", "slra_qk_rope"))]
    src, so = tmp_path / "older.c", tmp_path / "older.so"
    src.write_text("".join(f"int {n}(void) {{ return {slra.ABI_VERSION}; }}\n" for n in older))
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(so), str(src)], check=True)
    monkeypatch.setattr(slra, "_lib", None)
    monkeypatch.setattr(slra, "LIB_PATH", str(so))
    with pytest.raises(RuntimeError, match="older than this binding.*slra_qk_rope_fwd"):
        slra.lib()
